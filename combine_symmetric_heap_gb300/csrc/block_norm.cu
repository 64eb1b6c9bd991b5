// block_norm.cu -- the norms before and after a block, fused with the block's
// gate, dropout and residual scale; forward and backward.
//
//   n = o * rstd_o * w_post          rstd_o = (mean(o^2) + eps)^-1/2
//   y = x + scale * drop(act(gate) * n)
//   h = y * rstd_y * w_pre           rstd_y = (mean(y^2) + eps)^-1/2
//
// o is the block's output, x the residual stream, y the stream after the
// block, h the input of the next block.  Backward, with the stream's gradient
// dy and h's gradient dh, yn = y rstd_y, on = o rstd_o, m = scale * drop:
//   dx = dy + rstd_y (dh w_pre - yn mean(dh w_pre yn))
//   dn = m act(gate) dx;   do = rstd_o (dn w_post - on mean(dn w_post on))
//   dw_pre = sum dh yn,  dw_post = sum dn on,  dgate = act'(gate) sum m dx on w_post
// (sums over rows; the gate's over the rows that share it).
//
// Every row tensor is read once and written once; the dropout mask is recomputed
// from its counter; a row's sums come from one block reduction (the backward's
// two row means too: mean(dn w_post on) is linear in the first mean).  Three
// kernels each way, by the rows' length and alignment: staged (16-byte vectors,
// up to 8192 columns), odd (rows off 16-byte boundaries, up to 8192 columns) and
// general (any length, the row walked again out of L2).
//
// Measured (bf16, dropout 0.1, a GB300 whose copy rate is 6.69 TB/s): forward
// with both norms, 16384 x 4096, 129 us (4.2 TB/s; 89 us and 6.1 TB/s without
// dropout): a row's mask is made between its arrival and its sums, on the row's
// critical path (the dropout kernel, which has no such path, makes as many words
// in 67 us); backward, 8192 x 7168, 197 us (3.6 TB/s; 136 us and 5.2 TB/s without
// dropout), for the same reason and by the latency of a row's chain: its 57 KB a
// row and 16 columns' sums a thread leave an SM one block.  Rows off 16-byte boundaries: forward 16384 x 4095
// 219 us, backward 8192 x 7167 300 us.
#include <algorithm>

#include "rows_dev.cuh"

namespace symmoe {
namespace norm {

using namespace rows;

enum Act : int { ACT_NONE = 0, ACT_SIGMOID = 1, ACT_TANH = 2 };

// A row's address: rows and strides are 32-bit (one multiply-add of 64 bits)
template <typename T>
__device__ __forceinline__ const T *at(const void *p, int row, int ld) {
  return reinterpret_cast<const T *>(p) + (int64_t)row * ld;
}
template <typename T>
__device__ __forceinline__ T *at(void *p, int row, int ld) {
  return reinterpret_cast<T *>(p) + (int64_t)row * ld;
}

struct Fwd {
  const void *x, *o, *w_post, *w_pre, *gate;
  void *y, *h;
  float *rstd_post, *rstd_pre;
  int ldx, ldo, ldy, ldh, ldg;  // elements
  int rows, per_gate;           // per_gate: rows that share a gate row
  int gates, cols, act, post_norm;
  float scale, eps;
  int drop;
  Random rnd;
  int split;  // work items, as in Bwd
  int per_item;
};

struct Bwd {
  const void *dy, *dh, *y, *o, *w_post, *w_pre, *gate;
  const float *rstd_post, *rstd_pre;
  void *dx, *dout, *dw_pre, *dw_post, *dgate;
  float *ws;  // partial sums
  int ld_dy, ld_dh, ldy, ldo, ldg, ld_dx, ld_do, ld_dg;
  int rows, per_gate;
  int gates, cols, act, post_norm;
  float scale;
  int drop;
  Random rnd;
  // work items: `per_item` rows of a gate's rows; items = gates * split
  int split;
  int per_item;
};

__device__ __forceinline__ float activate(int act, float g) {
  if (act == ACT_SIGMOID) return __fdividef(1.f, 1.f + __expf(-g));
  if (act == ACT_TANH) return tanhf(g);
  return g;
}
__device__ __forceinline__ float slope(int act, float g) {
  if (act == ACT_SIGMOID) {
    const float s = __fdividef(1.f, 1.f + __expf(-g));
    return s * (1.f - s);
  }
  if (act == ACT_TANH) {
    const float t = tanhf(g);
    return 1.f - t * t;
  }
  return 1.f;
}

// Forward for rows of any length: the row is walked once for each sum and once
// to write (out of L2 after the first time).  V = 1: single elements, the row's
// dropout mask made once into shared memory.
template <typename T, int V>
__global__ void __launch_bounds__(1024) block_norm_kernel(const Fwd p) {
  extern __shared__ uint8_t mask[];
  __shared__ float buf[64];
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const float inv = 1.f / p.cols;
  int turn = 0;
  auto each = [&](auto &&f) {  // f(c) for this thread's vectors
    for (int c = (int)threadIdx.x * V; c < p.cols; c += blockDim.x * V) f(c);
  };
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T *x = at<T>(p.x, r, p.ldx), *o = p.o ? at<T>(p.o, r, p.ldo) : nullptr;
    const T *gate = p.gate ? at<T>(p.gate, r / p.per_gate, p.ldg) : nullptr;
    const T *w_post = reinterpret_cast<const T *>(p.w_post), *w_pre = reinterpret_cast<const T *>(p.w_pre);
    if (V == 1 && p.drop) {
      __syncthreads();  // the last row's mask has been read
      fill_mask(p.rnd, (uint64_t)r * p.cols, p.cols, mask, threadIdx.x, blockDim.x);
      __syncthreads();
    }
    float rstd_o = 1.f;
    if (o && p.post_norm) {
      float s[1] = {0.f};
      each([&](int c) {
        float v[V];
        load<T, V>(o + c, v);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += v[i] * v[i];
      });
      group_sums<1>(s, buf, warp, warps, turn);
      rstd_o = rsqrtf(s[0] * inv + p.eps);
      if (threadIdx.x == 0 && p.rstd_post) p.rstd_post[r] = rstd_o;
    }
    // y = x + scale * drop(act(gate) * n) for V columns
    auto stream = [&](int c, float(&y)[V]) {
      load<T, V>(x + c, y);
      if (!o) return;
      float f[V], t[V];
      load<T, V>(o + c, f);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] *= rstd_o * p.scale;
      if (w_post) {
        load<T, V>(w_post + c, t);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= t[i];
      }
      if (gate) {
        load<T, V>(gate + c, t);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= activate(p.act, t[i]);
      }
      if (p.drop) {
        if (V == 1) t[0] = mask[c] ? p.rnd.keep_scale : 0.f;
        else keep_factors<V>(p.rnd, (uint64_t)r * p.cols + c, t);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = t[i] != 0.f ? f[i] * t[i] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] += f[i];
    };
    float rstd_y = 0.f;
    if (p.h || p.rstd_pre) {
      float s[1] = {0.f};
      each([&](int c) {
        float v[V];
        stream(c, v);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += v[i] * v[i];
      });
      group_sums<1>(s, buf, warp, warps, turn);
      rstd_y = rsqrtf(s[0] * inv + p.eps);
      if (threadIdx.x == 0 && p.rstd_pre) p.rstd_pre[r] = rstd_y;
    }
    each([&](int c) {  // each column is read before it is written: y may be x
      float v[V], w[V];
      stream(c, v);
      if (p.y) store<T, V>(at<T>(p.y, r, p.ldy) + c, v);
      if (!p.h) return;
      if (w_pre) load<T, V>(w_pre + c, w);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= w_pre ? rstd_y * w[i] : rstd_y;
      store<T, V>(at<T>(p.h, r, p.ldh) + c, v);
    });
  }
}

// Backward for rows of any length: a block takes work items (a run of rows that
// share a gate row), one row at a time, walking it once for the sums and once
// for the results; the column sums live in the block's partial sums in the
// workspace and are joined by sum_partials_kernel in a fixed order.
template <typename T, int V>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(const Bwd p) {
  __shared__ float buf[2 * 32 * 3];
  extern __shared__ uint8_t mask[];  // V = 1: which elements of the row are kept
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const int items = p.gates * p.split;
  const float inv = 1.f / p.cols;
  int turn = 0;
  // workspace: [gridDim][cols] dw_pre, the same for dw_post, [items][cols] gate
  float *ws_pre = p.ws + (int64_t)blockIdx.x * p.cols;
  float *ws_post = p.ws + ((int64_t)gridDim.x + blockIdx.x) * p.cols;
  float *ws_gate = p.ws + 2 * (int64_t)gridDim.x * p.cols;
  const T *w_pre = reinterpret_cast<const T *>(p.w_pre), *w_post = reinterpret_cast<const T *>(p.w_post);

  auto each = [&](auto &&f) {  // f(c) for this thread's vectors
    for (int c = (int)threadIdx.x * V; c < p.cols; c += blockDim.x * V) f(c);
  };
  each([&](int c) {
#pragma unroll
    for (int i = 0; i < V; ++i) ws_pre[c + i] = ws_post[c + i] = 0.f;
  });

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t gi = item / p.split, first = gi * p.per_gate;
    const int64_t begin = first + (item % p.split) * p.per_item;
    const int64_t end = min(begin + p.per_item, first + p.per_gate);
    const T *gate = p.gate ? reinterpret_cast<const T *>(p.gate) + gi * p.ldg : nullptr;
    float *gate_sum = ws_gate + (int64_t)item * p.cols;
    if (p.dgate)
      each([&](int c) {
#pragma unroll
        for (int i = 0; i < V; ++i) gate_sum[c + i] = 0.f;
      });

    for (int64_t r = begin; r < end; ++r) {
      const T *dy = p.dy ? reinterpret_cast<const T *>(p.dy) + r * p.ld_dy : nullptr;
      const T *dh = p.dh ? reinterpret_cast<const T *>(p.dh) + r * p.ld_dh : nullptr;
      const T *y = p.dh ? reinterpret_cast<const T *>(p.y) + r * p.ldy : nullptr;
      const T *o = p.o ? reinterpret_cast<const T *>(p.o) + r * p.ldo : nullptr;
      const float ry = p.dh ? p.rstd_pre[r] : 0.f;
      const float ro = p.o && p.post_norm ? p.rstd_post[r] : 1.f;
      if (V == 1 && p.drop) {
        __syncthreads();  // the last row's mask has been read
        fill_mask(p.rnd, (uint64_t)r * p.cols, p.cols, mask, threadIdx.x, blockDim.x);
        __syncthreads();
      }
      // per column: yn, dx without its mean term (g0), on, the factor m * act
      // from dx to dn, and m alone (for the gate's gradient)
      auto columns = [&](int c, float(&yn)[V], float(&g0)[V], float(&hv)[V], float(&on)[V], float(&fa)[V],
                         float(&fm)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) yn[i] = g0[i] = hv[i] = on[i] = fa[i] = fm[i] = 0.f;
        if (dy) load<T, V>(dy + c, g0);
        if (dh) {
          load<T, V>(y + c, yn);
          load<T, V>(dh + c, hv);
          float w[V];
#pragma unroll
          for (int i = 0; i < V; ++i) w[i] = 1.f;
          if (w_pre) load<T, V>(w_pre + c, w);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            yn[i] *= ry;
            g0[i] += ry * hv[i] * w[i];
          }
        }
        if (o) {
          load<T, V>(o + c, on);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            on[i] *= ro;
            fm[i] = p.scale;
          }
          if (p.drop) {
            float k[V];
            if (V == 1) k[0] = mask[c] ? p.rnd.keep_scale : 0.f;
            else keep_factors<V>(p.rnd, (uint64_t)r * p.cols + c, k);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              fm[i] *= k[i];
              if (k[i] == 0.f && !(ro > 0.f)) on[i] = 0.f;  // as clear_dropped does
            }
          }
          if (gate) {
            float g[V];
            load<T, V>(gate + c, g);
#pragma unroll
            for (int i = 0; i < V; ++i) fa[i] = fm[i] * activate(p.act, g[i]);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) fa[i] = fm[i];
          }
        }
      };
      auto post_weight = [&](int c, float(&w)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = 1.f;
        if (w_post) load<T, V>(w_post + c, w);
      };
      // sums over the row: dh w_pre yn;  g0 q;  yn q  with q = m act w_post on
      float s[3] = {0.f, 0.f, 0.f};
      each([&](int c) {
        float yn[V], g0[V], hv[V], on[V], fa[V], fm[V], w[V];
        columns(c, yn, g0, hv, on, fa, fm);
        post_weight(c, w);
        float wp[V];
#pragma unroll
        for (int i = 0; i < V; ++i) wp[i] = 1.f;
        if (dh && w_pre) load<T, V>(w_pre + c, wp);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float q = fa[i] != 0.f ? fa[i] * w[i] * on[i] : 0.f;
          s[0] += hv[i] * wp[i] * yn[i];
          s[1] += g0[i] * q;
          s[2] += yn[i] * q;
        }
      });
      group_sums<3>(s, buf, warp, warps, turn);
      const float m1 = ry * s[0] * inv;                                  // dx = g0 - yn * m1
      const float m2 = p.post_norm ? (s[1] - m1 * s[2]) * inv : 0.f;     // mean(dn w_post on)
      each([&](int c) {
        float yn[V], g0[V], hv[V], on[V], fa[V], fm[V], w[V];
        columns(c, yn, g0, hv, on, fa, fm);
        post_weight(c, w);
        float dov[V], dxv[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float dx = g0[i] - yn[i] * m1;
          // a dropped element passes nothing on, whatever its values
          const float dn = fa[i] != 0.f ? dx * fa[i] : 0.f;
          const float dg = fm[i] != 0.f ? dx * fm[i] * on[i] * w[i] : 0.f;
          dxv[i] = dx;
          dov[i] = ro * (dn * w[i] - (p.post_norm ? on[i] * m2 : 0.f));
          hv[i] *= yn[i];
          fa[i] = fa[i] != 0.f ? dn * on[i] : 0.f;
          fm[i] = dg;
        }
        if (p.dx) store<T, V>(reinterpret_cast<T *>(p.dx) + r * p.ld_dx + c, dxv);
        if (p.dout) store<T, V>(reinterpret_cast<T *>(p.dout) + r * p.ld_do + c, dov);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          ws_pre[c + i] += hv[i];
          ws_post[c + i] += fa[i];
          if (p.dgate) gate_sum[c + i] += fm[i];
        }
      });
    }
    if (p.dgate)
      each([&](int c) {
        float t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = gate_sum[c + i];
        if (p.split == 1) {  // this block saw all rows of the gate row
          float g[V];
          load<T, V>(gate + c, g);
#pragma unroll
          for (int i = 0; i < V; ++i) t[i] *= slope(p.act, g[i]);
          store<T, V>(reinterpret_cast<T *>(p.dgate) + gi * p.ld_dg + c, t);
        }
      });
  }
}

// ---------------------------------------------------------------------------
// Staged kernels: rows in 16-byte vectors, at most 8192 columns.  A block walks
// work items (runs of rows that share a gate row); a thread holds 8 or 16
// columns and copies its own vectors of the next rows into its own shared
// memory (cp.async, a few rows deep), so no barrier guards the copies.  What a
// column needs for every row stays with its thread for the item's rows: the
// activated gate in registers, the weights in shared memory.
//
// With rows of a few thousand columns these kernels are bound by the latency
// of a row's chain (read, reduce, finish) as much as by bytes: one reduction a
// row, four sums at a time; no branches in the inner loops (tensors that are
// not there, and columns past the row's end, are zeros in shared memory, the
// weights ones); addresses that are constants from a row's start.
// ---------------------------------------------------------------------------
constexpr int STAGED_COLS = 8192;
constexpr int STAGED_SMEM = 220 * 1024;  // of a block, at most (the odd kernels too)
constexpr int MASK_SMEM = 65536;         // a row's mask bytes in the general kernels, at most
// A gate row shared by this few rows is copied along with each of them.
constexpr int GATE_WITH_ROWS = 4;

// A block's rows in the order of its work items
struct Walk {
  int per_gate, per_item, row, end, item, items, split;
  __device__ Walk(int per_gate_, int per_item_, int gates, int split_)
      : per_gate(per_gate_), per_item(per_item_), item(blockIdx.x), items(gates * split_), split(split_) {
    open();
  }
  __device__ void open() {  // the item's rows (every item has some)
    const int g = item / split, first = g * per_gate;
    row = first + (item - g * split) * per_item;
    end = min(row + per_item, first + per_gate);
  }
  __device__ bool live() const { return item < items; }
  __device__ void next() {
    if (++row < end) return;
    item += gridDim.x;
    open();
  }
};

// A thread's columns: NG groups of 8.  16-bit types: a group is one 16-byte
// vector; fp32: two.  A thread's vectors lie a warp's width apart in a row
// (NEAR: constant offsets) or a block's, and MAXT words of 16 bytes apart in
// shared memory.  Near is faster where instructions count (16384 x 4096 forward
// 133 -> 129 us, 8192 x 7168 backward 198 -> 192, 150 -> 144 without dropout), but
// not in the forward without dropout, which is bound by memory (89 -> 94 us).
template <typename T, int NG_, int MAXT_, bool NEAR>
struct Columns {
  static constexpr int NG = NG_, MAXT = MAXT_;
  static constexpr int PER = sizeof(T) / 2;  // vectors of a group
  static constexpr int NV = NG * PER;
  static constexpr int W = 16 / sizeof(T);   // columns of a vector
  static __device__ __forceinline__ int vector(int j) {
    const int t = threadIdx.x;
    return (NEAR ? t / 32 * (32 * NV) + (t & 31) + 32 * j : t + j * (int)blockDim.x) * W;
  }
  static __device__ __forceinline__ int quad(int g, int k) { return vector(g * PER + k / (W / 4)) + 4 * (k % (W / 4)); }
  // place of vector j of array a in a row's shared memory, in bytes
  static __device__ __forceinline__ constexpr int place(int a, int j) { return (a * NV + j) * MAXT * 16; }
  static __host__ __device__ constexpr int row_bytes(int arrays) { return arrays * NV * MAXT * 16; }
};
// A group's 8 values of one array: two quads
template <typename C, typename T>
struct Eight {
  uint4 v[C::PER];
  __device__ __forceinline__ Eight(const char *p, int g) {
#pragma unroll
    for (int j = 0; j < C::PER; ++j) v[j] = *reinterpret_cast<const uint4 *>(p + C::place(0, g * C::PER + j));
  }
  __device__ __forceinline__ void quad(int k, float (&f)[4]) const {
    if constexpr (sizeof(T) == 4) {
      unpack<T, 4>(v[k], f);
    } else {
      const float2 a = Elem<T>::get2(k ? v[0].z : v[0].x), b = Elem<T>::get2(k ? v[0].w : v[0].y);
      f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    }
  }
};
// Quads' results as whole 16-byte stores
template <typename T>
struct Writer {
  typename Quad<T>::Word first;
  __device__ __forceinline__ void put(int k, T *row, int col, int cols, const float (&f)[4]) {
    const typename Quad<T>::Word w = Quad<T>::put(f);
    if constexpr (sizeof(T) == 4) {
      if (col < cols) *reinterpret_cast<uint4 *>(row + col) = w;
    } else {
      if (k == 0) first = w;
      else if (col < cols) *reinterpret_cast<uint4 *>(row + col - 4) = make_uint4(first.x, first.y, w.x, w.y);
    }
  }
};
// scale * act(gate) * w_post of a quad
template <typename T>
__device__ __forceinline__ void factor_of(float scale, int act, const void *gate, const T *w_post, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = scale;
  if (gate) {
    float g[4];
    Quad<T>::get(gate, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] *= activate(act, g[i]);
  }
  if (w_post) {
    float w[4];
    Quad<T>::get(w_post, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] *= w[i];
  }
}
// zeros in a thread's part of the rows, w_pre (or ones) in its fixed part
template <typename C, typename T>
__device__ __forceinline__ void prepare_rows(char *row0, char *end, char *fixed, const T *w_pre, int cols) {
  for (char *q = row0; q < end; q += C::MAXT * 16) *reinterpret_cast<uint4 *>(q) = make_uint4(0, 0, 0, 0);
  float one[Elem<T>::VEC];
#pragma unroll
  for (int i = 0; i < Elem<T>::VEC; ++i) one[i] = 1.f;
#pragma unroll
  for (int j = 0; j < C::NV; ++j)
    *reinterpret_cast<uint4 *>(fixed + C::place(0, j)) =
        w_pre && C::vector(j) < cols ? *reinterpret_cast<const uint4 *>(w_pre + C::vector(j)) : pack<T, Elem<T>::VEC>(one);
}
// Bit 8g + 4k + i: is element i of quad k of group first + g of row r kept?
template <typename C, int N>
__device__ __forceinline__ uint32_t row_mask(const Random &rnd, int r, int cols, int first) {
  uint64_t block[2 * N];
#pragma unroll
  for (int g = 0; g < N; ++g)
#pragma unroll
    for (int k = 0; k < 2; ++k) block[2 * g + k] = ((uint64_t)r * cols + C::quad(first + g, k)) >> 2;
  return kept_bits<2 * N>(rnd, block);
}
__device__ __forceinline__ void wait_oldest(int ahead) {
  if (ahead == 3) cp_async_wait<2>();
  else if (ahead == 2) cp_async_wait<1>();
  else cp_async_wait<0>();
}

// Forward.  With q = scale drop act(gate) w_post o, y = x + rstd_o q, so the sum
// of y^2 comes from the same reduction as rstd_o's: with f = rstd_o (and the
// kept elements' scale), y^2 sums to s1 + f (2 s2 + f s3) of the sums of x^2, x q
// and q^2.  That does not hold where the parts cancel (y shorter than a third of
// them), where a product of values not yet normalised left the range of fp32, or
// where so small ones vanished (each by less than 2^-149) that f^2 brings back.
// Such a row is read again and taken in the definition's order.
__device__ __forceinline__ bool sums_hold(float yy, const float (&s)[4], float f, float inv, float eps) {
  return yy <= 3e38f && yy >= 0.1f * (s[1] + f * (f * s[3])) && f * (f + 2.f) * 1.5e-38f <= yy * inv + eps;
}
template <typename T, bool DROP, int NG, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 384 ? 2 : 0)
    block_norm_staged_kernel(const Fwd p, int gate_with_rows, int ahead_rows) {
  using C = Columns<T, NG, MAXT, DROP>;
  extern __shared__ __align__(16) char smem[];
  __shared__ float buf[2 * 128];
  enum { X, O, GATE };
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const int row_step = C::row_bytes(2 + gate_with_rows);
  char *const row0 = smem + threadIdx.x * 16, *const row_end = row0 + ahead_rows * row_step, *const fixed = row_end;
  const float inv = 1.f / p.cols;
  const T *w_post = reinterpret_cast<const T *>(p.w_post);
  prepare_rows<C, T>(row0, row_end, fixed, reinterpret_cast<const T *>(p.w_pre), p.cols);
  Walk ahead(p.per_gate, p.per_item, p.gates, p.split), now = ahead;
  auto fetch = [&](char *to) {  // the next row
    if (ahead.live()) {
      const int r = ahead.row;
#pragma unroll
      for (int j = 0; j < C::NV; ++j) {
        const int c = C::vector(j);
        if (c < p.cols) {
          cp_async16(to + C::place(X, j), at<T>(p.x, r, p.ldx) + c);
          if (p.o) cp_async16(to + C::place(O, j), at<T>(p.o, r, p.ldo) + c);
          if (gate_with_rows) cp_async16(to + C::place(GATE, j), at<T>(p.gate, ahead.item / p.split, p.ldg) + c);
        }
      }
      ahead.next();
    }
    cp_async_commit();
  };
  for (char *to = row0; to != row_end; to += row_step) fetch(to);
  char *row = row0;
  float factor[NG][2][4];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int i = 0; i < 8; ++i) factor[g][i / 4][i % 4] = 0.f;
  int half = 0, item = -1;
  for (; now.live(); now.next()) {
    const int r = now.row;
    if (now.item != item && !gate_with_rows) {
      item = now.item;
      const T *gate = p.gate ? at<T>(p.gate, item / p.split, p.ldg) : nullptr;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = C::quad(g, k);
          if (c < p.cols) factor_of<T>(p.scale, p.act, gate ? gate + c : nullptr, w_post ? w_post + c : nullptr, factor[g][k]);
        }
    }
    wait_oldest(ahead_rows);
    if (gate_with_rows)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = C::quad(g, k);
          const char *gate = row + C::place(GATE, g * C::PER + k / (C::W / 4)) + 4 * (k % (C::W / 4)) * (int)sizeof(T);
          if (c < p.cols) factor_of<T>(p.scale, p.act, gate, w_post ? w_post + c : nullptr, factor[g][k]);
        }
    // sums of o^2, x^2, x q, q^2
    float x[NG][2][4], q[NG][2][4], s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t kept = DROP ? row_mask<C, 1>(p.rnd, r, p.cols, g) : 0u;
      const Eight<C, T> x8(row + C::place(X, 0), g), o8(row + C::place(O, 0), g);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float ov[4];
        x8.quad(k, x[g][k]);
        o8.quad(k, ov);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool keep = !DROP || ((kept >> (4 * k + i)) & 1u);
          const float xv = x[g][k][i], qv = keep ? ov[i] * factor[g][k][i] : 0.f;
          q[g][k][i] = qv;
          s[0] += ov[i] * ov[i];
          s[1] += xv * xv;
          s[2] += xv * qv;
          s[3] += qv * qv;
        }
      }
    }
    fetch(row);
    row = row + row_step == row_end ? row0 : row + row_step;
    block_sums4(s, buf, warp, warps, half);
    const float rstd_o = p.post_norm ? rsqrtf(s[0] * inv + p.eps) : 1.f;
    const float f = DROP ? rstd_o * p.rnd.keep_scale : rstd_o;
    float yy = s[1] + f * (2.f * s[2] + f * s[3]);
    if (sums_hold(yy, s, f, inv, p.eps)) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[g][i / 4][i % 4] += f * q[g][i / 4][i % 4];  // y
    } else {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t kept = DROP ? row_mask<C, 1>(p.rnd, r, p.cols, g) : 0u;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = C::quad(g, k);
          float xv[4] = {0.f, 0.f, 0.f, 0.f}, ov[4] = {0.f, 0.f, 0.f, 0.f};
          if (c < p.cols) {
            Quad<T>::get(at<T>(p.x, r, p.ldx) + c, xv);
            if (p.o) Quad<T>::get(at<T>(p.o, r, p.ldo) + c, ov);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool keep = !DROP || ((kept >> (4 * k + i)) & 1u);
            const float y = xv[i] + (keep ? ov[i] * f * factor[g][k][i] : 0.f);
            x[g][k][i] = y;
            t[0] += y * y;
          }
        }
      }
      block_sums4(t, buf, warp, warps, half);
      yy = t[0];
    }
    const float rstd_y = rsqrtf(yy * inv + p.eps);
    if (threadIdx.x == 0) {
      if (p.rstd_post) p.rstd_post[r] = rstd_o;
      if (p.rstd_pre) p.rstd_pre[r] = rstd_y;
    }
    Writer<T> out;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (p.y)
#pragma unroll
        for (int k = 0; k < 2; ++k) out.put(k, at<T>(p.y, r, p.ldy), C::quad(g, k), p.cols, x[g][k]);
      if (!p.h) continue;
      const Eight<C, T> w8(fixed, g);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float w[4];
        w8.quad(k, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] *= x[g][k][i] * rstd_y;
        out.put(k, at<T>(p.h, r, p.ldh), C::quad(g, k), p.cols, w);
      }
    }
  }
}

// An infinite o makes its row's rstd 0 and itself NaN when normalised: where it is
// dropped, a zero in its place (this thread's elements of the row's copy)
template <typename C, typename T>
__device__ __forceinline__ void clear_dropped(char *p, uint32_t kept) {
#pragma unroll 1
  for (int e = 0; e < 8 * C::NG; ++e)
    if (!((kept >> e) & 1u))
      *reinterpret_cast<T *>(p + C::place(0, e / C::W) + e % C::W * (int)sizeof(T)) = Elem<T>::put(0.f);
}

// Backward.  Per column the block keeps two sums: of dh yn (dw_pre), and over
// an item's rows S = sum drop dx on, from which both dw_post = sum over gates
// of scale act S and dgate = scale act' w_post S follow.  o is normalised before
// anything else multiplies it, so that rows of any size stay in range; without
// the norm after the block (POST) o is in S only.  (One block an SM, said
// to the compiler: it takes all registers and reads further ahead, 134 against 144
// us at 8192 x 7168 without dropout.  With dropout it had them anyway.)
template <typename T, bool DROP, bool POST, int NG, int MAXT>
__global__ void __launch_bounds__(MAXT, !DROP && NG == 2 ? 1 : 0)
    block_norm_bwd_staged_kernel(const Bwd p, int gate_with_rows, int ahead_rows) {
  using C = Columns<T, NG, MAXT, true>;
  extern __shared__ __align__(16) char smem[];
  __shared__ float buf[2 * 128];
  enum { DY, DH, Y, O, GATE };
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const int row_step = C::row_bytes(4 + gate_with_rows);
  char *const row0 = smem + threadIdx.x * 16, *const row_end = row0 + ahead_rows * row_step, *const fixed = row_end;
  // dw_post's sums over the items: quad k of group g at post[(2g + k) * MAXT]
  float4 *const post = reinterpret_cast<float4 *>(fixed + C::row_bytes(1));
  const float inv = 1.f / p.cols;
  const T *w_post = reinterpret_cast<const T *>(p.w_post);
  prepare_rows<C, T>(row0, row_end, fixed, reinterpret_cast<const T *>(p.w_pre), p.cols);
  Walk ahead(p.per_gate, p.per_item, p.gates, p.split), now = ahead, soon = ahead;
  auto fetch = [&](char *to) {  // the next row
    if (ahead.live()) {
      const int r = ahead.row;
#pragma unroll
      for (int j = 0; j < C::NV; ++j) {
        const int c = C::vector(j);
        if (c < p.cols) {
          if (p.dy) cp_async16(to + C::place(DY, j), at<T>(p.dy, r, p.ld_dy) + c);
          if (p.dh) {
            cp_async16(to + C::place(DH, j), at<T>(p.dh, r, p.ld_dh) + c);
            cp_async16(to + C::place(Y, j), at<T>(p.y, r, p.ldy) + c);
          }
          if (p.o) cp_async16(to + C::place(O, j), at<T>(p.o, r, p.ldo) + c);
          if (gate_with_rows) cp_async16(to + C::place(GATE, j), at<T>(p.gate, ahead.item / p.split, p.ldg) + c);
        }
      }
      ahead.next();
    }
    cp_async_commit();
  };
  // 1 / rms of the next row, read one row ahead
  float ry = 0.f, ro = 1.f;
  auto read_rstd = [&](const Walk &w) {
    if (!w.live()) return;
    if (p.dh) ry = p.rstd_pre[w.row];
    if (POST && p.o) ro = p.rstd_post[w.row];
  };
  for (char *to = row0; to != row_end; to += row_step) fetch(to);
  read_rstd(soon);
  char *row = row0;
  float factor[NG][2][4], a_pre[NG][2][4], a_s[NG][2][4];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      post[(2 * g + k) * MAXT] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) factor[g][k][i] = a_pre[g][k][i] = a_s[g][k][i] = 0.f;
    }
  auto gate_row = [&](int item) { return p.gate ? at<T>(p.gate, item / p.split, p.ldg) : nullptr; };
  // an item's S goes to dw_post's sums and to the gate's gradient (directly
  // where the item is all of the gate row's rows)
  auto flush = [&](int item) {
    if (!p.o || item < 0) return;
    const T *gate = gate_row(item);
    Writer<T> out;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = C::quad(g, k);
        if (c < p.cols) {
          float gv[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {1.f, 1.f, 1.f, 1.f}, s[4];
          if (gate) Quad<T>::get(gate + c, gv);
          if (w_post) Quad<T>::get(w_post + c, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[i] = p.scale * a_s[g][k][i];
            a_s[g][k][i] = 0.f;
            w[i] *= s[i];
            if (gate) s[i] *= activate(p.act, gv[i]);
          }
          float4 sum = post[(2 * g + k) * MAXT];
          sum.x += s[0], sum.y += s[1], sum.z += s[2], sum.w += s[3];
          post[(2 * g + k) * MAXT] = sum;
          if (!p.dgate) continue;
          if (p.split == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] *= slope(p.act, gv[i]);
            out.put(k, at<T>(p.dgate, item, p.ld_dg), c, p.cols, w);
          } else {
            float *sums = p.ws + 2 * (int64_t)gridDim.x * p.cols + (int64_t)item * p.cols;
            *reinterpret_cast<float4 *>(sums + c) = make_float4(w[0], w[1], w[2], w[3]);
          }
        }
      }
  };
  // a group's values of a row; yn, dx without its mean term and dh of a quad
  // (s0 += dh w_pre yn)
  struct Row {
    Eight<C, T> dy, dh, y, o, w;
    __device__ __forceinline__ Row(const char *row, const char *fixed, int g)
        : dy(row + C::place(DY, 0), g), dh(row + C::place(DH, 0), g), y(row + C::place(Y, 0), g),
          o(row + C::place(O, 0), g), w(fixed, g) {}
    __device__ __forceinline__ void front(int k, float ry, float (&yn)[4], float (&g0)[4], float (&hv)[4],
                                          float &s0) const {
      float wv[4];
      dy.quad(k, g0);
      dh.quad(k, hv);
      y.quad(k, yn);
      w.quad(k, wv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        yn[i] *= ry;
        const float t = hv[i] * wv[i];
        g0[i] += ry * t;
        s0 += t * yn[i];
      }
    }
  };
  const float ks = DROP ? p.rnd.keep_scale : 1.f;
  int half = 0, item = -1;
  for (; now.live(); now.next()) {
    const int r = now.row;
    const float cy = ry, co = ro;  // this row's
    soon.next();
    read_rstd(soon);
    if (now.item != item) {
      flush(item);
      item = now.item;
      const T *gate = gate_row(item);
      if (!gate_with_rows)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int c = C::quad(g, k);
            if (c < p.cols) factor_of<T>(p.scale, p.act, gate ? gate + c : nullptr, w_post ? w_post + c : nullptr, factor[g][k]);
          }
    }
    wait_oldest(ahead_rows);
    if (gate_with_rows)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = C::quad(g, k);
          const char *gate = row + C::place(GATE, g * C::PER + k / (C::W / 4)) + 4 * (k % (C::W / 4)) * (int)sizeof(T);
          if (c < p.cols) factor_of<T>(p.scale, p.act, gate, w_post ? w_post + c : nullptr, factor[g][k]);
        }
    // all groups' blocks of words side by side (a group at a time: 203 against
    // 197 us; the forward, with fewer registers to spare, gains from that)
    const uint32_t kept = DROP ? row_mask<C, C::NG>(p.rnd, r, p.cols, 0) : 0u;  // bit 8g + 4k + i
    if (DROP && POST && !(co > 0.f)) clear_dropped<C, T>(row + C::place(O, 0), kept);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const Row in(row, fixed, g);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float yn[4], g0[4], hv[4], ov[4];
        in.front(k, cy, yn, g0, hv, s[0]);
        in.o.quad(k, ov);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool keep = !DROP || ((kept >> (8 * g + 4 * k + i)) & 1u);
          if (POST) {
            const float q = keep ? factor[g][k][i] * (ov[i] * co) : 0.f;
            s[1] += g0[i] * q;
            s[2] += yn[i] * q;
          }
        }
      }
    }
    block_sums4(s, buf, warp, warps, half);
    // The row is read from shared memory again: without this the compiler keeps its
    // values in registers over the reduction (100 instead of 76 a thread at 8 columns,
    // 8192 x 1024 44 us instead of 33; at 8192 x 7168 152 instead of 136).
    asm volatile("" ::: "memory");
    const float m1 = cy * s[0] * inv;  // dx = g0 - yn * m1
    const float m2 = ks * (s[1] - m1 * s[2]) * inv;  // mean(dn w_post on)
    Writer<T> out_x, out_o;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const Row in(row, fixed, g);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = C::quad(g, k);
        float yn[4], g0[4], hv[4], ov[4], unused = 0.f;
        in.front(k, cy, yn, g0, hv, unused);
        in.o.quad(k, ov);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a_pre[g][k][i] += hv[i] * yn[i];
          g0[i] -= yn[i] * m1;  // dx
          // a dropped element passes nothing on, whatever its values
          const bool keep = !DROP || ((kept >> (8 * g + 4 * k + i)) & 1u);
          const float d = keep ? g0[i] * ks : 0.f;  // drop dx
          if constexpr (POST) {
            const float on = ov[i] * co;
            a_s[g][k][i] += d * on;
            ov[i] = co * (d * factor[g][k][i] - on * m2);
          } else {
            a_s[g][k][i] += d * (keep ? ov[i] : 0.f);
            ov[i] = d * factor[g][k][i];
          }
        }
        if (p.dx) out_x.put(k, at<T>(p.dx, r, p.ld_dx), c, p.cols, g0);
        if (p.dout) out_o.put(k, at<T>(p.dout, r, p.ld_do), c, p.cols, ov);
      }
    }
    fetch(row);
    row = row + row_step == row_end ? row0 : row + row_step;
  }
  flush(item);
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = C::quad(g, k);
      if (c < p.cols) {
        const float(&a)[4] = a_pre[g][k];
        const float4 sum = post[(2 * g + k) * MAXT];
        if (gridDim.x == 1) {  // the sums are whole: no launch to add partials
          const float b[4] = {sum.x, sum.y, sum.z, sum.w};
          if (p.dw_pre) *reinterpret_cast<typename Quad<T>::Word *>(reinterpret_cast<T *>(p.dw_pre) + c) = Quad<T>::put(a);
          if (p.dw_post) *reinterpret_cast<typename Quad<T>::Word *>(reinterpret_cast<T *>(p.dw_post) + c) = Quad<T>::put(b);
          continue;
        }
        if (p.dw_pre)
          *reinterpret_cast<float4 *>(p.ws + (int64_t)blockIdx.x * p.cols + c) = make_float4(a[0], a[1], a[2], a[3]);
        if (p.dw_post) *reinterpret_cast<float4 *>(p.ws + ((int64_t)gridDim.x + blockIdx.x) * p.cols + c) = sum;
      }
    }
}

// ---------------------------------------------------------------------------
// Rows that start off a 16-byte boundary (odd lengths, sliced tensors), up to
// 8192 columns: the staged kernels' work with 8 single elements a thread, 32
// apart (a warp's are 256 in a row, their offsets constants).  A row is copied as the 16-byte words that it lies in,
// up to three rows ahead, and lies in shared memory as far from a boundary as
// in memory; here any thread may read what another one copied, so a thread's
// copies of the next row are waited for before a barrier of this row.  A row's
// dropout mask is made a row ahead too, each block of words once.  Columns past
// the row's end are zeros in shared memory, as in the staged kernels.
//
// Bound by instructions: an element at a time, bf16 and fp32 take the same time
// (218 and 229 us forward at 16384 x 4095, 144 and 174 without dropout).  With
// the next row's elements loaded into registers instead, 307 us, and 757 against
// 335 backward; columns a block's width apart, whose addresses are computed, 250
// and 423.
// ---------------------------------------------------------------------------
constexpr int ODD_EACH = 8, ODD_COLS = ODD_EACH * 1024;
// This thread's first column; the others follow 32 apart
__device__ __forceinline__ int odd_first() {
  return (int)threadIdx.x / 32 * (32 * ODD_EACH) + ((int)threadIdx.x & 31);
}
// A row of any alignment in shared memory, and a row's mask bytes, for `threads` threads
template <typename T>
__host__ __device__ constexpr int odd_pitch(int threads) {
  return ODD_EACH * threads * (int)sizeof(T) + 16;
}
__host__ __device__ constexpr int odd_mask_pitch(int threads) { return ODD_EACH * threads + 8; }
// How far from a 16-byte boundary row r starts
template <typename T>
__device__ __forceinline__ int odd_shift(const void *p, int r, int ld) {
  return p ? (int)(reinterpret_cast<uintptr_t>(at<T>(p, r, ld)) & 15) : 0;
}
// 16 bytes to shared memory, of which `n` are read and the rest are zeros
__device__ __forceinline__ void cp_async16_part(char *to, const char *from, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(n) : "memory");
}
// Copy row r of `cols` elements to `to` + its shift.  The first word begins up to
// 15 bytes before the row: memory of the same allocation, since those begin on
// 16-byte boundaries (it is read, never used).  The last word is cut at the row's
// end, and zeros follow where a row of another shift may have ended.
template <typename T>
__device__ __forceinline__ void odd_copy(char *to, const void *p, int r, int ld, int cols, int pitch) {
  if (!p) return;
  const int shift = odd_shift<T>(p, r, ld), bytes = shift + cols * (int)sizeof(T);
  const char *from = reinterpret_cast<const char *>(at<T>(p, r, ld)) - shift;
  for (int i = 16 * (int)threadIdx.x; i < min(bytes + 16, pitch); i += 16 * (int)blockDim.x) {
    const int n = max(0, min(16, bytes - i));
    cp_async16_part(to + i, n ? from + i : from, n);
  }
}
// Which elements of row r are kept, a byte each: element c at mask[(r cols) mod 4 + c]
__device__ __forceinline__ void odd_mask(const Random &rnd, int r, int cols, uint8_t *mask) {
  const uint64_t first = (uint64_t)r * cols;
  const int blocks = ((int)(first & 3) + cols + 3) / 4, T = blockDim.x;
  for (int b = threadIdx.x; b < blocks; b += 2 * T) {
    const uint64_t block[2] = {(first >> 2) + b, (first >> 2) + b + T};
    const uint32_t kept = kept_bits<2>(rnd, block);
    // bit i of four to byte i
    reinterpret_cast<uint32_t *>(mask)[b] = ((kept & 15u) * 0x00204081u) & 0x01010101u;
    if (b + T < blocks) reinterpret_cast<uint32_t *>(mask)[b + T] = ((kept >> 4) * 0x00204081u) & 0x01010101u;
  }
}
template <typename T>
__device__ __forceinline__ float odd_get(const char *row, int c) {
  return Elem<T>::get(*reinterpret_cast<const T *>(row + c * (int)sizeof(T)));
}
// Zeros in the rows
__device__ __forceinline__ void odd_clear(char *rows, const char *end) {
  for (char *q = rows + 16 * threadIdx.x; q < end; q += 16 * blockDim.x)
    *reinterpret_cast<uint4 *>(q) = make_uint4(0, 0, 0, 0);
  __syncthreads();
}
// scale * act(gate) * w_post of this thread's columns (`gate`: in memory, or with the row)
template <typename T>
__device__ __forceinline__ void odd_factors(float scale, int act, const T *gate, const T *w_post, int cols,
                                            float (&f)[ODD_EACH]) {
  float g[ODD_EACH], w[ODD_EACH];
#pragma unroll
  for (int e = 0; e < ODD_EACH; ++e) {
    const int c = odd_first() + 32 * e;
    g[e] = gate && c < cols ? Elem<T>::get(gate[c]) : 0.f;
    w[e] = w_post && c < cols ? Elem<T>::get(w_post[c]) : 1.f;
  }
#pragma unroll
  for (int e = 0; e < ODD_EACH; ++e) f[e] = scale * (gate ? activate(act, g[e]) : 1.f) * w[e];
}

template <typename T, bool DROP>
__global__ void __launch_bounds__(1024) block_norm_odd_kernel(const Fwd p, int gate_with_rows, int ahead_rows) {
  constexpr int NE = ODD_EACH;
  extern __shared__ __align__(16) char smem[];
  __shared__ float buf[2 * 128];
  enum { X, O, GATE };
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, pitch = odd_pitch<T>(blockDim.x);
  const int row_step = (2 + gate_with_rows) * pitch;
  char *const row_end = smem + ahead_rows * row_step;
  T *const w = reinterpret_cast<T *>(row_end);
  uint8_t *const masks = reinterpret_cast<uint8_t *>(row_end + pitch);
  const int mask_pitch = odd_mask_pitch(blockDim.x);
  const float inv = 1.f / p.cols;
  const T *w_post = reinterpret_cast<const T *>(p.w_post);
  auto col = [&](int e) { return odd_first() + 32 * e; };
  Walk now(p.per_gate, p.per_item, p.gates, p.split), soon = now, ahead = now;
  odd_clear(smem, row_end);
  auto fetch = [&](char *to) {  // the next row
    if (ahead.live()) {
      odd_copy<T>(to + X * pitch, p.x, ahead.row, p.ldx, p.cols, pitch);
      odd_copy<T>(to + O * pitch, p.o, ahead.row, p.ldo, p.cols, pitch);
      if (gate_with_rows) odd_copy<T>(to + GATE * pitch, p.gate, ahead.item / p.split, p.ldg, p.cols, pitch);
      ahead.next();
    }
    cp_async_commit();
  };
  for (char *to = smem; to != row_end; to += row_step) fetch(to);
  if (DROP) odd_mask(p.rnd, soon.row, p.cols, masks);
  float factor[NE];
#pragma unroll
  for (int e = 0; e < NE; ++e) factor[e] = 0.f;
  const T *w_pre = reinterpret_cast<const T *>(p.w_pre);
#pragma unroll
  for (int e = 0; e < NE; ++e) w[col(e)] = w_pre && col(e) < p.cols ? w_pre[col(e)] : Elem<T>::put(1.f);
  wait_oldest(ahead_rows);
  __syncthreads();
  char *row = smem;
  int half = 0, item = -1, side = 0;
  for (; now.live(); now.next()) {
    const int r = now.row;
    if (now.item != item || gate_with_rows) {
      item = now.item;
      const T *gate = p.gate ? at<T>(p.gate, item / p.split, p.ldg) : nullptr;
      if (gate_with_rows)
        gate = reinterpret_cast<const T *>(row + GATE * pitch + odd_shift<T>(p.gate, item / p.split, p.ldg));
      odd_factors<T>(p.scale, p.act, gate, w_post, p.cols, factor);
    }
    const char *rx = row + X * pitch + odd_shift<T>(p.x, r, p.ldx), *ro = row + O * pitch + odd_shift<T>(p.o, r, p.ldo);
    const uint8_t *mask = masks + side * mask_pitch + (((uint32_t)r * (uint32_t)p.cols) & 3u);
    float y[NE], q[NE], s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const float o = odd_get<T>(ro, col(e));
      y[e] = odd_get<T>(rx, col(e));
      q[e] = !DROP || mask[col(e)] ? o * factor[e] : 0.f;
      s[0] += o * o;
      s[1] += y[e] * y[e];
      s[2] += y[e] * q[e];
      s[3] += q[e] * q[e];
    }
    soon.next();
    side ^= 1;
    if (DROP && soon.live()) odd_mask(p.rnd, soon.row, p.cols, masks + side * mask_pitch);
    if (ahead_rows > 1) wait_oldest(ahead_rows - 1);  // the next row
    block_sums4(s, buf, warp, warps, half);
    if (warps == 1) __syncwarp();
    fetch(row);
    row = row + row_step == row_end ? smem : row + row_step;
    const float rstd_o = p.post_norm ? rsqrtf(s[0] * inv + p.eps) : 1.f;
    const float f = DROP ? rstd_o * p.rnd.keep_scale : rstd_o;
    float yy = s[1] + f * (2.f * s[2] + f * s[3]);
    if (sums_hold(yy, s, f, inv, p.eps)) {
#pragma unroll
      for (int e = 0; e < NE; ++e) y[e] += f * q[e];
    } else {
      // (the row's mask bytes may be the next row's by now: its words are made again)
      float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const int c = col(e);
        const bool in = c < p.cols;
        const float xv = in ? Elem<T>::get(at<T>(p.x, r, p.ldx)[c]) : 0.f;
        const float ov = in && p.o ? Elem<T>::get(at<T>(p.o, r, p.ldo)[c]) : 0.f;
        float k[1] = {1.f};
        if (DROP) keep_factors<1>(p.rnd, (uint64_t)r * p.cols + c, k);
        y[e] = xv + (k[0] != 0.f ? ov * f * factor[e] : 0.f);
        t[0] += y[e] * y[e];
      }
      block_sums4(t, buf, warp, warps, half);
      yy = t[0];
    }
    const float rstd_y = rsqrtf(yy * inv + p.eps);
    if (threadIdx.x == 0) {
      if (p.rstd_post) p.rstd_post[r] = rstd_o;
      if (p.rstd_pre) p.rstd_pre[r] = rstd_y;
    }
    if (p.y) {
      T *py = at<T>(p.y, r, p.ldy);
#pragma unroll
      for (int e = 0; e < NE; ++e)
        if (col(e) < p.cols) py[col(e)] = Elem<T>::put(y[e]);
    }
    if (p.h) {
      T *ph = at<T>(p.h, r, p.ldh);
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const T v = Elem<T>::put(y[e] * rstd_y * Elem<T>::get(w[col(e)]));
        if (col(e) < p.cols) ph[col(e)] = v;
      }
    }
    if (ahead_rows == 1) {
      cp_async_wait<0>();
      __syncthreads();
    }
  }
}

template <typename T, bool DROP>
__global__ void __launch_bounds__(1024) block_norm_bwd_odd_kernel(const Bwd p, int gate_with_rows, int ahead_rows) {
  constexpr int NE = ODD_EACH;
  extern __shared__ __align__(16) char smem[];
  __shared__ float buf[2 * 128];
  enum { DY, DH, Y, O, GATE };
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, pitch = odd_pitch<T>(blockDim.x);
  const int row_step = (4 + gate_with_rows) * pitch;
  char *const row_end = smem + ahead_rows * row_step;
  T *const w = reinterpret_cast<T *>(row_end);
  float *const post = reinterpret_cast<float *>(row_end + pitch);  // dw_post's sums over the items
  uint8_t *const masks = reinterpret_cast<uint8_t *>(post + NE * blockDim.x);
  const int mask_pitch = odd_mask_pitch(blockDim.x);
  const float inv = 1.f / p.cols;
  const T *w_post = reinterpret_cast<const T *>(p.w_post);
  auto col = [&](int e) { return odd_first() + 32 * e; };
  Walk now(p.per_gate, p.per_item, p.gates, p.split), soon = now, ahead = now;
  odd_clear(smem, row_end);
  const T *w_pre = reinterpret_cast<const T *>(p.w_pre);
  for (int c = threadIdx.x; c < NE * (int)blockDim.x; c += blockDim.x)
    w[c] = w_pre && c < p.cols ? w_pre[c] : Elem<T>::put(1.f);
  auto fetch = [&](char *to) {  // the next row
    if (ahead.live()) {
      const int r = ahead.row;
      odd_copy<T>(to + DY * pitch, p.dy, r, p.ld_dy, p.cols, pitch);
      if (p.dh) {
        odd_copy<T>(to + DH * pitch, p.dh, r, p.ld_dh, p.cols, pitch);
        odd_copy<T>(to + Y * pitch, p.y, r, p.ldy, p.cols, pitch);
      }
      odd_copy<T>(to + O * pitch, p.o, r, p.ldo, p.cols, pitch);
      if (gate_with_rows) odd_copy<T>(to + GATE * pitch, p.gate, ahead.item / p.split, p.ldg, p.cols, pitch);
      ahead.next();
    }
    cp_async_commit();
  };
  float ry = 0.f, ro = 1.f;  // 1 / rms of the next row
  auto read_rstd = [&]() {
    if (!soon.live()) return;
    if (p.dh) ry = p.rstd_pre[soon.row];
    if (p.o && p.post_norm) ro = p.rstd_post[soon.row];
  };
  for (char *to = smem; to != row_end; to += row_step) fetch(to);
  read_rstd();
  if (DROP) odd_mask(p.rnd, soon.row, p.cols, masks);
  float factor[NE], a_pre[NE], a_s[NE];
#pragma unroll
  for (int e = 0; e < NE; ++e) factor[e] = a_pre[e] = a_s[e] = post[col(e)] = 0.f;
  auto flush = [&](int item) {  // as in the staged kernel
    if (!p.o || item < 0) return;
    const T *gate = p.gate ? at<T>(p.gate, item / p.split, p.ldg) : nullptr;
    float g[NE], d[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      g[e] = gate && col(e) < p.cols ? Elem<T>::get(gate[col(e)]) : 0.f;
      d[e] = w_post && col(e) < p.cols ? Elem<T>::get(w_post[col(e)]) : 1.f;
    }
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const float s = p.scale * a_s[e];
      a_s[e] = 0.f;
      d[e] *= s;
      post[col(e)] += gate ? activate(p.act, g[e]) * s : s;
    }
    if (!p.dgate) return;
    if (p.split == 1) {
      T *to = at<T>(p.dgate, item, p.ld_dg);
#pragma unroll
      for (int e = 0; e < NE; ++e)
        if (col(e) < p.cols) to[col(e)] = Elem<T>::put(d[e] * slope(p.act, g[e]));
    } else {
      float *to = p.ws + 2 * (int64_t)gridDim.x * p.cols + (int64_t)item * p.cols;
#pragma unroll
      for (int e = 0; e < NE; ++e)
        if (col(e) < p.cols) to[col(e)] = d[e];
    }
  };
  wait_oldest(ahead_rows);
  __syncthreads();
  const float ks = DROP ? p.rnd.keep_scale : 1.f;
  char *row = smem;
  int half = 0, item = -1, side = 0;
  for (; now.live(); now.next()) {
    const int r = now.row;
    const float cy = ry, co = ro;
    soon.next();
    read_rstd();
    if (now.item != item) flush(item);
    if (now.item != item || gate_with_rows) {
      item = now.item;
      const T *gate = p.gate ? at<T>(p.gate, item / p.split, p.ldg) : nullptr;
      if (gate_with_rows)
        gate = reinterpret_cast<const T *>(row + GATE * pitch + odd_shift<T>(p.gate, item / p.split, p.ldg));
      odd_factors<T>(p.scale, p.act, gate, w_post, p.cols, factor);
    }
    const char *rdy = row + DY * pitch + odd_shift<T>(p.dy, r, p.ld_dy), *rdh = row + DH * pitch;
    const char *ryy = row + Y * pitch, *rov = row + O * pitch + odd_shift<T>(p.o, r, p.ldo);
    if (p.dh) rdh += odd_shift<T>(p.dh, r, p.ld_dh), ryy += odd_shift<T>(p.y, r, p.ldy);
    const uint8_t *mask = masks + side * mask_pitch + (((uint32_t)r * (uint32_t)p.cols) & 3u);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t kept = 0u;
    if (DROP && !(co > 0.f))  // as clear_dropped does; no other thread reads these elements
      for (int e = 0; e < NE; ++e)
        if (!mask[col(e)]) *reinterpret_cast<T *>(const_cast<char *>(rov) + col(e) * (int)sizeof(T)) = Elem<T>::put(0.f);
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int c = col(e);
      const float yn = odd_get<T>(ryy, c) * cy, t = odd_get<T>(rdh, c) * Elem<T>::get(w[c]);
      const float g0 = odd_get<T>(rdy, c) + cy * t;
      if (DROP) kept |= (uint32_t)mask[c] << e;
      const float q = !DROP || ((kept >> e) & 1u) ? factor[e] * (odd_get<T>(rov, c) * co) : 0.f;
      s[0] += t * yn;
      s[1] += g0 * q;
      s[2] += yn * q;
    }
    side ^= 1;
    if (DROP && soon.live()) odd_mask(p.rnd, soon.row, p.cols, masks + side * mask_pitch);
    block_sums4(s, buf, warp, warps, half);
    const float m1 = cy * s[0] * inv;
    const float m2 = p.post_norm ? ks * (s[1] - m1 * s[2]) * inv : 0.f;
    T *const dx_row = p.dx ? at<T>(p.dx, r, p.ld_dx) : nullptr, *const do_row = p.dout ? at<T>(p.dout, r, p.ld_do) : nullptr;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int c = col(e);
      const bool in = c < p.cols;
      const float hv = odd_get<T>(rdh, c), yn = odd_get<T>(ryy, c) * cy, on = odd_get<T>(rov, c) * co;
      const float dx = odd_get<T>(rdy, c) + cy * (hv * Elem<T>::get(w[c])) - yn * m1;
      a_pre[e] += hv * yn;
      const bool keep = !DROP || ((kept >> e) & 1u);
      const float d = keep ? dx * ks : 0.f;
      if (keep) a_s[e] += d * on;
      const T vx = Elem<T>::put(dx), vo = Elem<T>::put(co * (d * factor[e] - (p.post_norm ? on * m2 : 0.f)));
      if (in && dx_row) dx_row[c] = vx;
      if (in && do_row) do_row[c] = vo;
    }
    if (ahead_rows > 1) wait_oldest(ahead_rows - 1);  // the next row
    __syncthreads();  // it has come, and this one has been read
    fetch(row);
    row = row + row_step == row_end ? smem : row + row_step;
    if (ahead_rows == 1) {
      cp_async_wait<0>();
      __syncthreads();
    }
  }
  flush(item);
#pragma unroll
  for (int e = 0; e < NE; ++e)
    if (col(e) < p.cols) {
      const int c = col(e);
      if (gridDim.x == 1) {  // the sums are whole: no launch to add partials
        if (p.dw_pre) reinterpret_cast<T *>(p.dw_pre)[c] = Elem<T>::put(a_pre[e]);
        if (p.dw_post) reinterpret_cast<T *>(p.dw_post)[c] = Elem<T>::put(post[c]);
        continue;
      }
      if (p.dw_pre) p.ws[(int64_t)blockIdx.x * p.cols + c] = a_pre[e];
      if (p.dw_post) p.ws[((int64_t)gridDim.x + blockIdx.x) * p.cols + c] = post[c];
    }
}

// Column sums of the partials: y 0 dw_pre, 1 dw_post, 2 + g the gate rows.
// A block adds 32 columns with 32 warps: warp w takes partials w, w + 32, ...,
// four in flight, then the warps' sums are added in order.  (Eight warps, one
// load in flight: 30 of the backward's 62 us at 8192 rows of 1024.)
constexpr int SUM_WARPS = 32;
template <typename T>
__global__ void __launch_bounds__(32 * SUM_WARPS) sum_partials_kernel(const Bwd p, int blocks) {
  __shared__ float part[SUM_WARPS][33];
  pdl_wait();  // the partials
  const int which = blockIdx.y;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x / 32;
  const bool is_gate = which >= 2;
  void *out = which == 0 ? p.dw_pre : which == 1 ? p.dw_post : p.dgate;
  if (!out || (is_gate && p.split == 1)) return;
  const float *from = p.ws + (which == 0 ? 0 : which == 1 ? (int64_t)blocks * p.cols
                                                          : 2 * (int64_t)blocks * p.cols +
                                                                (int64_t)(which - 2) * p.split * p.cols);
  const int n = is_gate ? p.split : blocks;
  float s = 0.f;
  if (c < p.cols) {
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = w; i < n; i += 4 * SUM_WARPS)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * SUM_WARPS < n) t[k] += from[(int64_t)(i + k * SUM_WARPS) * p.cols + c];
    s = (t[0] + t[1]) + (t[2] + t[3]);
  }
  part[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w != 0 || c >= p.cols) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < SUM_WARPS; ++i) s += part[i][threadIdx.x];
  if (is_gate) {
    const int64_t gi = which - 2;
    s *= slope(p.act, Elem<T>::get(reinterpret_cast<const T *>(p.gate)[gi * p.ldg + c]));
    reinterpret_cast<T *>(p.dgate)[gi * p.ld_dg + c] = Elem<T>::put(s);
  } else {
    reinterpret_cast<T *>(out)[c] = Elem<T>::put(s);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Threads for rows of `cols` elements, `each` a thread: whole warps
static int threads_of(int cols, int each) { return ((cols + each - 1) / each + 31) / 32 * 32; }

// A staged block: 8 columns a thread in rows of up to 2048 columns (blocks of up
// to 64 or 256 threads, which sets the shared memory's layout), 16 beyond.  At
// 4096 columns, forward, three resident blocks of 256 threads instead of two
// were slower (102 against 88 us without dropout, the same with it), so were 8
// columns a thread (94 against 88, 145 against 133).  Beyond 4096 columns, two
// blocks of up to 384 threads at 80 registers instead of one, in the forward of
// 16-bit types (`two`): 8192 x 5120 92 against 107 us, 61 against 74 without
// dropout; 8192 x 6144 101 against 109.  fp32 loses (6144: 145 against 137), the
// backward too (5120: 170 against 158): too few registers.
struct StagedShape {
  int groups, max_threads, threads, per_sm;
};
static StagedShape staged_shape(int cols, bool two) {
  StagedShape s;
  s.groups = cols <= 2048 ? 1 : 2;
  s.max_threads = cols <= 512 ? 64 : cols <= 2048 ? 256 : two && cols > 4096 && cols <= 6144 ? 384 : 512;
  s.threads = (cols + 256 * s.groups - 1) / (256 * s.groups) * 32;
  // resident blocks an SM: by their registers, 768 threads of small blocks, else 512
  s.per_sm = std::max(1, (s.groups == 1 || s.max_threads == 384 ? 768 : 512) / s.threads);
  return s;
}
static int64_t staged_blocks(int64_t rows, const StagedShape &s, int num_sms) {
  return std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms * s.per_sm));
}
// An odd rows' blocks: 64 registers a thread, so up to 1024 threads an SM
static int odd_threads(int cols) { return threads_of(cols, ODD_EACH); }
static int odd_per_sm(int threads) { return std::max(1, 1024 / threads); }
static int64_t odd_blocks(int64_t rows, int threads, int num_sms) {
  return std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms * odd_per_sm(threads)));
}
// As launch_staged; a block also has its 1 KB for the sums and 1 KB reserved
template <typename P>
static cudaError_t launch_odd(void (*kern)(P, int, int), const P &p, int arrays, int pitch, size_t fixed, int blocks,
                              int threads, cudaStream_t st) {
  const size_t room = STAGED_SMEM / odd_per_sm(threads) - 2048;
  const int with_rows = p.gate && p.per_gate <= GATE_WITH_ROWS && fixed + (size_t)pitch * (arrays + 1) <= room;
  const size_t row = (size_t)pitch * (arrays + with_rows);
  const int ahead = room < fixed + 2 * row ? 1 : room < fixed + 3 * row ? 2 : 3;
  const size_t bytes = fixed + ahead * row;
  const cudaError_t err = allow_smem(kern, STAGED_SMEM);
  if (err != cudaSuccess) return err;
  kern<<<blocks, threads, bytes, st>>>(p, with_rows, ahead);
  return cudaGetLastError();
}
// f(group count, threads' limit) as types
template <bool TWO, typename F>
static auto with_shape(const StagedShape &s, F f) {
  using std::integral_constant;
  if (s.max_threads == 64) return f(integral_constant<int, 1>{}, integral_constant<int, 64>{});
  if (s.max_threads == 256) return f(integral_constant<int, 1>{}, integral_constant<int, 256>{});
  if constexpr (TWO)
    if (s.max_threads == 384) return f(integral_constant<int, 2>{}, integral_constant<int, 384>{});
  return f(integral_constant<int, 2>{}, integral_constant<int, 512>{});
}
// Launch with rows copied ahead (up to three, as many as leave room for the
// resident blocks) and, where it fits, the gate copied with them
template <typename C, typename P>
static cudaError_t launch_staged(void (*kern)(P, int, int), const P &p, int arrays, size_t fixed, bool gate, int blocks,
                                 const StagedShape &s, cudaStream_t st) {
  const int with_rows = gate && fixed + C::row_bytes(arrays + 1) <= STAGED_SMEM;
  const size_t row = C::row_bytes(arrays + with_rows), room = STAGED_SMEM / s.per_sm;
  const int ahead = room < fixed + 2 * row ? 1 : room < fixed + 3 * row ? 2 : 3;
  const size_t bytes = fixed + ahead * row;
  const cudaError_t err = allow_smem(kern, STAGED_SMEM);
  if (err != cudaSuccess) return err;
  kern<<<blocks, s.threads, bytes, st>>>(p, with_rows, ahead);
  return cudaGetLastError();
}
// Split of a gate row's rows into items, about one for each block and none
// without rows (each leaves a partial sum that is added)
static int64_t split_of(int64_t gates, int64_t per_gate, int64_t blocks) {
  if (gates >= blocks) return 1;
  const int64_t split = std::max<int64_t>(1, std::min<int64_t>(per_gate, blocks / gates));
  const int64_t per_item = (per_gate + split - 1) / split;
  return (per_gate + per_item - 1) / per_item;
}

template <typename T, int V>
static cudaError_t fwd(Fwd p, int num_sms, cudaStream_t st) {
  if constexpr (V > 1) {
    if (p.cols <= STAGED_COLS) {
      constexpr bool two = sizeof(T) == 2;
      const StagedShape s = staged_shape(p.cols, two);
      const int64_t most = staged_blocks(p.rows, s, num_sms);
      p.split = (int)split_of(p.gates, p.per_gate, most);
      p.per_item = (p.per_gate + p.split - 1) / p.split;
      const int blocks = (int)std::min<int64_t>(most, (int64_t)p.gates * p.split);
      return with_shape<two>(s, [&](auto groups, auto threads) {
        using C = Columns<T, decltype(groups)::value, decltype(threads)::value, true>;  // (for the sizes)
        return launch_staged<C, Fwd>(p.drop ? block_norm_staged_kernel<T, true, C::NG, C::MAXT>
                                            : block_norm_staged_kernel<T, false, C::NG, C::MAXT>,
                                     p, 2, C::row_bytes(1), p.gate && p.per_gate <= GATE_WITH_ROWS, blocks, s, st);
      });
    }
  } else {
    if (p.cols <= ODD_COLS) {
      const int threads = odd_threads(p.cols);
      const int64_t most = odd_blocks(p.rows, threads, num_sms);
      p.split = (int)split_of(p.gates, p.per_gate, most);
      p.per_item = (p.per_gate + p.split - 1) / p.split;
      const int blocks = (int)std::min<int64_t>(most, (int64_t)p.gates * p.split), pitch = odd_pitch<T>(threads);
      return launch_odd(p.drop ? block_norm_odd_kernel<T, true> : block_norm_odd_kernel<T, false>, p, 2, pitch,
                        pitch + (p.drop ? 2 * odd_mask_pitch(threads) : 0), blocks, threads, st);
    }
  }
  auto kern = block_norm_kernel<T, V>;
  const size_t smem = V == 1 && p.drop ? p.cols : 0;
  const cudaError_t err = allow_smem(kern, MASK_SMEM);
  if (err != cudaSuccess) return err;
  kern<<<std::min(p.rows, num_sms * 2), 1024, smem, st>>>(p);
  return cudaGetLastError();
}

// The backward's launch: threads and blocks for rows in vectors of V
struct BwdPlan {
  bool staged, odd;  // neither: the general kernel
  int threads;
  int64_t blocks;
};
static BwdPlan plan_bwd(int64_t rows, int cols, int V, int num_sms) {
  if (V > 1 && cols <= STAGED_COLS) {
    const StagedShape s = staged_shape(cols, false);
    return BwdPlan{true, false, s.threads, staged_blocks(rows, s, num_sms)};
  }
  if (V == 1 && cols <= ODD_COLS) {
    const int threads = odd_threads(cols);
    return BwdPlan{false, true, threads, odd_blocks(rows, threads, num_sms)};
  }
  return BwdPlan{false, false, 512, std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms * 2))};
}

template <typename T, int V>
static cudaError_t bwd(Bwd p, int num_sms, cudaStream_t st) {
  const BwdPlan plan = plan_bwd(p.rows, p.cols, V, num_sms);
  p.split = (int)split_of(p.gates, p.per_gate, plan.blocks);
  p.per_item = (p.per_gate + p.split - 1) / p.split;
  const int blocks = (int)std::min<int64_t>(plan.blocks, (int64_t)p.gates * p.split);
  cudaError_t err = cudaSuccess;
  if constexpr (V > 1) {
    if (plan.staged) {
      const StagedShape s = staged_shape(p.cols, false);
      err = with_shape<false>(s, [&](auto groups, auto threads) {
        using C = Columns<T, decltype(groups)::value, decltype(threads)::value, true>;  // (for the sizes)
        auto kern = p.post_norm ? (p.drop ? block_norm_bwd_staged_kernel<T, true, true, C::NG, C::MAXT>
                                          : block_norm_bwd_staged_kernel<T, false, true, C::NG, C::MAXT>)
                                : (p.drop ? block_norm_bwd_staged_kernel<T, true, false, C::NG, C::MAXT>
                                          : block_norm_bwd_staged_kernel<T, false, false, C::NG, C::MAXT>);
        return launch_staged<C, Bwd>(kern, p, 4, C::row_bytes(1) + 2 * C::NG * C::MAXT * 16,
                                     p.gate && p.per_gate <= GATE_WITH_ROWS, blocks, s, st);
      });
      if (err != cudaSuccess) return err;
    } else {
      block_norm_bwd_kernel<T, V><<<blocks, plan.threads, 0, st>>>(p);
    }
  } else {
    if (plan.odd) {
      const int pitch = odd_pitch<T>(plan.threads);
      err = launch_odd(p.drop ? block_norm_bwd_odd_kernel<T, true> : block_norm_bwd_odd_kernel<T, false>, p, 4, pitch,
                       pitch + 4 * ODD_EACH * plan.threads + (p.drop ? 2 * odd_mask_pitch(plan.threads) : 0), blocks,
                       plan.threads, st);
      if (err != cudaSuccess) return err;
    } else {
      const size_t smem = p.drop ? p.cols : 0;
      err = allow_smem(block_norm_bwd_kernel<T, 1>, MASK_SMEM);
      if (err != cudaSuccess) return err;
      block_norm_bwd_kernel<T, 1><<<blocks, plan.threads, smem, st>>>(p);
    }
  }
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const bool gates = p.dgate && p.split > 1;
  if (!((plan.staged || plan.odd) && blocks == 1) && (p.dw_pre || p.dw_post || gates))
    err = launch_pdl(sum_partials_kernel<T>, dim3((p.cols + 31) / 32, 2 + (gates ? p.gates : 0)),
                     dim3(32 * SUM_WARPS), 0, st, p,
                     blocks);
  return err;
}

// 16-byte vectors where every row of every tensor starts on their boundary
static bool vec_ok(std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> lds, int cols, int64_t es) {
  for (const void *q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) % 16) return false;
  for (int64_t l : lds)
    if (l * es % 16) return false;
  return cols * es % 16 == 0;
}

}  // namespace norm

// bytes of partial sums, an upper bound over the types and alignments
size_t block_norm_workspace(int64_t rows, int cols, int64_t gates, int num_sms) {
  using namespace norm;
  size_t best = 0;
  for (int V : {1, 4, 8}) {
    const BwdPlan plan = plan_bwd(rows, cols, V, num_sms);
    const int64_t split = gates ? split_of(gates, rows / gates, plan.blocks) : 1;
    // gate partials: where several blocks share a gate row, or (rows beyond
    // the register budget) the sums live in memory
    const int64_t items = gates && (split > 1 || (!plan.staged && !plan.odd)) ? gates * split : 0;
    best = std::max(best, (size_t)(2 * plan.blocks + items) * cols * sizeof(float));
  }
  return best;
}

cudaError_t launch_block_norm(const sym_block_norm &a, int num_sms, cudaStream_t st) {
  using namespace norm;
  Fwd p = {};
  p.x = a.x, p.o = a.o, p.w_post = a.w_post, p.w_pre = a.w_pre, p.gate = a.gate, p.y = a.y, p.h = a.h;
  p.rstd_post = a.rstd_post, p.rstd_pre = a.rstd_pre;
  p.ldx = (int)a.ld_x, p.ldo = (int)a.ld_o, p.ldy = (int)a.ld_y, p.ldh = (int)a.ld_h, p.ldg = (int)a.ld_gate;
  p.rows = (int)a.rows, p.gates = a.gate ? (int)a.gate_rows : 1;
  p.per_gate = p.rows / p.gates;
  // no norm after a block that is not there (its rstd would be 1 / sqrt(eps),
  // infinite at eps = 0)
  p.cols = a.cols, p.act = a.gate_act, p.post_norm = a.o && !(a.flags & SYM_NORM_NO_POST);
  p.scale = a.scale, p.eps = a.eps, p.drop = a.p > 0;
  p.rnd = make_random(a.seed, a.offset, a.p);
  const int64_t es = a.dtype == SYM_FP32 ? 4 : 2;
  const bool vec = vec_ok({p.x, p.o, p.w_post, p.w_pre, p.gate, p.y, p.h},
                          {p.ldx, p.o ? p.ldo : 0, p.y ? p.ldy : 0, p.h ? p.ldh : 0, p.gate ? p.ldg : 0}, p.cols, es);
  if (a.dtype == SYM_BF16) return vec ? fwd<__nv_bfloat16, 8>(p, num_sms, st) : fwd<__nv_bfloat16, 1>(p, num_sms, st);
  if (a.dtype == SYM_FP16) return vec ? fwd<__half, 8>(p, num_sms, st) : fwd<__half, 1>(p, num_sms, st);
  return vec ? fwd<float, 4>(p, num_sms, st) : fwd<float, 1>(p, num_sms, st);
}

cudaError_t launch_block_norm_bwd(const sym_block_norm &a, const sym_block_norm_grad &b, int num_sms,
                                  cudaStream_t st) {
  using namespace norm;
  Bwd p = {};
  p.dy = b.dy, p.dh = b.dh, p.y = a.y, p.o = a.o, p.w_post = a.w_post, p.w_pre = a.w_pre, p.gate = a.gate;
  p.rstd_post = a.rstd_post, p.rstd_pre = a.rstd_pre;
  p.dx = b.dx, p.dout = b.d_o, p.dw_pre = b.dw_pre, p.dw_post = b.dw_post, p.dgate = b.dgate;
  p.ws = reinterpret_cast<float *>(b.work);
  p.ld_dy = (int)b.ld_dy, p.ld_dh = (int)b.ld_dh, p.ldy = (int)a.ld_y, p.ldo = (int)a.ld_o, p.ldg = (int)a.ld_gate;
  p.ld_dx = (int)b.ld_dx, p.ld_do = (int)b.ld_do, p.ld_dg = (int)b.ld_dgate;
  p.rows = (int)a.rows, p.gates = a.gate ? (int)a.gate_rows : 1;
  p.per_gate = p.rows / p.gates;
  p.cols = a.cols, p.act = a.gate_act, p.post_norm = !(a.flags & SYM_NORM_NO_POST);
  p.scale = a.scale, p.drop = a.p > 0;
  p.rnd = make_random(a.seed, a.offset, a.p);
  const int64_t es = a.dtype == SYM_FP32 ? 4 : 2;
  const bool vec = vec_ok({p.dy, p.dh, p.dh ? p.y : nullptr, p.o, p.w_post, p.w_pre, p.gate, p.dx, p.dout, p.dgate, p.dw_pre,
                           p.dw_post},
                          {p.dy ? p.ld_dy : 0, p.dh ? p.ld_dh : 0, p.dh ? p.ldy : 0, p.o ? p.ldo : 0,
                           p.gate ? p.ldg : 0, p.dx ? p.ld_dx : 0, p.dout ? p.ld_do : 0, p.dgate ? p.ld_dg : 0},
                          p.cols, es);
  if (a.dtype == SYM_BF16) return vec ? bwd<__nv_bfloat16, 8>(p, num_sms, st) : bwd<__nv_bfloat16, 1>(p, num_sms, st);
  if (a.dtype == SYM_FP16) return vec ? bwd<__half, 8>(p, num_sms, st) : bwd<__half, 1>(p, num_sms, st);
  return vec ? bwd<float, 4>(p, num_sms, st) : bwd<float, 1>(p, num_sms, st);
}

}  // namespace symmoe
