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
// Both are bound by their bytes: every row tensor is read once and written
// once, one pass per row with the row held in registers (rows beyond the
// register budget are walked again out of L2).  The dropout mask is recomputed
// from its counter.  The backward's two row means are taken with one block
// reduction: mean(dn w_post on) is linear in the first mean.
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

// The stream after the block for V columns of a row: x + scale * drop(gate * n)
template <typename T, int V>
__device__ __forceinline__ void stream_after(const Fwd &p, const T *x, const float (&ov)[V], float rstd, const T *gate,
                                             int64_t row, int c, float (&yv)[V]) {
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = ov[i] * rstd;
  if (p.w_post) {
    float w[V];
    load<T, V>(reinterpret_cast<const T *>(p.w_post) + c, w);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] *= w[i];
  }
  if (gate) {
    float g[V];
    load<T, V>(gate + c, g);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] *= activate(p.act, g[i]);
  }
  if (p.drop) {
    float k[V];
    keep_factors<V>(p.rnd, (uint64_t)row * p.cols + c, k);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = k[i] != 0.f ? f[i] * k[i] : 0.f;
  }
  load<T, V>(x + c, yv);
#pragma unroll
  for (int i = 0; i < V; ++i) yv[i] += p.scale * f[i];
}

// Forward.  NV > 0: a thread keeps its NV vectors of the row in registers;
// NV = 0: any row length, the row is walked once per sum and once to write.
// blockDim (threads of a row, rows of a block).
template <typename T, int V, int NV>
__global__ void __launch_bounds__(1024) block_norm_kernel(const Fwd p) {
  extern __shared__ float buf[];
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  float *mine = buf + threadIdx.y * 64;
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const float inv = 1.f / p.cols;
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < p.rows; r0 += step) {
    const int64_t want = r0 + threadIdx.y;
    const bool live = want < p.rows;
    const int64_t r = live ? want : p.rows - 1;  // idle row groups follow along without writing
    const T *x = reinterpret_cast<const T *>(p.x) + r * p.ldx;
    const T *o = p.o ? reinterpret_cast<const T *>(p.o) + r * p.ldo : nullptr;
    const T *gate = p.gate ? reinterpret_cast<const T *>(p.gate) + (r / p.per_gate) * p.ldg : nullptr;
    T *y = p.y ? reinterpret_cast<T *>(p.y) + r * p.ldy : nullptr;
    T *h = p.h ? reinterpret_cast<T *>(p.h) + r * p.ldh : nullptr;
    constexpr int N = NV ? NV : 1;
    float yv[N][V];
    float rstd_o = 1.f;
    if (o && p.post_norm) {
      float s[1] = {0.f};
      if (NV) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int c = ((int)threadIdx.x + j * (int)blockDim.x) * V;
          if (c < p.cols) {
            load<T, V>(o + c, yv[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) s[0] += yv[j][i] * yv[j][i];
          }
        }
      } else {
        for (int c = (int)threadIdx.x * V; c < p.cols; c += blockDim.x * V) {
          float ov[V];
          load<T, V>(o + c, ov);
#pragma unroll
          for (int i = 0; i < V; ++i) s[0] += ov[i] * ov[i];
        }
      }
      group_sums<1>(s, mine, warp, warps, turn);
      rstd_o = rsqrtf(s[0] * inv + p.eps);
      if (live && threadIdx.x == 0 && p.rstd_post) p.rstd_post[r] = rstd_o;
    }
    // V columns of y from c on, o's values in ov where the row is in registers
    auto stream = [&](int c, const float(&ov)[V], float(&out)[V]) {
      if (!o) load<T, V>(x + c, out);
      else if (NV && p.post_norm) stream_after<T, V>(p, x, ov, rstd_o, gate, r, c, out);
      else {
        float fresh[V];
        load<T, V>(o + c, fresh);
        stream_after<T, V>(p, x, fresh, rstd_o, gate, r, c, out);
      }
    };
    float s[1] = {0.f};
    if (NV) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int c = ((int)threadIdx.x + j * (int)blockDim.x) * V;
        if (c < p.cols) {
          float t[V];
          stream(c, yv[j], t);
          if (y && live) store<T, V>(y + c, t);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            yv[j][i] = t[i];
            s[0] += t[i] * t[i];
          }
        }
      }
    } else if (h || p.rstd_pre) {
      for (int c = (int)threadIdx.x * V; c < p.cols; c += blockDim.x * V) {
        float t[V];
        stream(c, t, t);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += t[i] * t[i];
      }
    }
    float rstd_y = 0.f;
    if (h || p.rstd_pre) {
      group_sums<1>(s, mine, warp, warps, turn);
      rstd_y = rsqrtf(s[0] * inv + p.eps);
      if (live && threadIdx.x == 0 && p.rstd_pre) p.rstd_pre[r] = rstd_y;
    }
    auto finish = [&](int c, float(&t)[V]) {
      if (!h || !live) return;
      if (p.w_pre) {
        float w[V];
        load<T, V>(reinterpret_cast<const T *>(p.w_pre) + c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = t[i] * rstd_y * w[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] *= rstd_y;
      }
      store<T, V>(h + c, t);
    };
    if (NV) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int c = ((int)threadIdx.x + j * (int)blockDim.x) * V;
        if (c < p.cols) finish(c, yv[j]);
      }
    } else {
      for (int c = (int)threadIdx.x * V; c < p.cols; c += blockDim.x * V) {
        float t[V];
        stream(c, t, t);  // each column is read before it is written: y may be x
        if (y && live) store<T, V>(y + c, t);
        finish(c, t);
      }
    }
  }
}

// Backward.  A block takes work items (a run of rows that share a gate row),
// one row at a time; the column sums stay in registers over its rows (NV > 0)
// or in the block's partial sums in the workspace (NV = 0), and are joined by
// sum_partials_kernel in a fixed order.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(const Bwd p) {
  __shared__ float buf[2 * 32 * 3];
  constexpr int N = NV ? NV : 1;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const int items = p.gates * p.split;
  const float inv = 1.f / p.cols;
  int turn = 0;
  // workspace: [gridDim][cols] dw_pre, the same for dw_post, [items][cols] gate
  float *ws_pre = p.ws + (int64_t)blockIdx.x * p.cols;
  float *ws_post = p.ws + ((int64_t)gridDim.x + blockIdx.x) * p.cols;
  float *ws_gate = p.ws + 2 * (int64_t)gridDim.x * p.cols;
  float a_pre[N][V], a_post[N][V], a_gate[N][V];
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) a_pre[j][i] = a_post[j][i] = 0.f;
  const T *w_pre = reinterpret_cast<const T *>(p.w_pre), *w_post = reinterpret_cast<const T *>(p.w_post);

  auto each = [&](auto &&f) {  // f(j, c) for this thread's vectors
    if (NV) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int c = ((int)threadIdx.x + j * (int)blockDim.x) * V;
        if (c < p.cols) f(j, c);
      }
    } else {
      for (int c = (int)threadIdx.x * V; c < p.cols; c += blockDim.x * V) f(0, c);
    }
  };
  if (!NV)
    each([&](int, int c) {
#pragma unroll
      for (int i = 0; i < V; ++i) ws_pre[c + i] = ws_post[c + i] = 0.f;
    });

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t gi = item / p.split, first = gi * p.per_gate;
    const int64_t begin = first + (item % p.split) * p.per_item;
    const int64_t end = min(begin + p.per_item, first + p.per_gate);
    const T *gate = p.gate ? reinterpret_cast<const T *>(p.gate) + gi * p.ldg : nullptr;
    float *gate_sum = ws_gate + (int64_t)item * p.cols;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) a_gate[j][i] = 0.f;
    if (!NV && p.dgate)
      each([&](int, int c) {
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
            keep_factors<V>(p.rnd, (uint64_t)r * p.cols + c, k);
#pragma unroll
            for (int i = 0; i < V; ++i) fm[i] *= k[i];
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
      each([&](int, int c) {
        float yn[V], g0[V], hv[V], on[V], fa[V], fm[V], w[V];
        columns(c, yn, g0, hv, on, fa, fm);
        post_weight(c, w);
        float wp[V];
#pragma unroll
        for (int i = 0; i < V; ++i) wp[i] = 1.f;
        if (dh && w_pre) load<T, V>(w_pre + c, wp);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float q = fa[i] * w[i] * on[i];
          s[0] += hv[i] * wp[i] * yn[i];
          s[1] += g0[i] * q;
          s[2] += yn[i] * q;
        }
      });
      group_sums<3>(s, buf, warp, warps, turn);
      const float m1 = ry * s[0] * inv;                                  // dx = g0 - yn * m1
      const float m2 = p.post_norm ? (s[1] - m1 * s[2]) * inv : 0.f;     // mean(dn w_post on)
      each([&](int j, int c) {
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
          dov[i] = ro * (dn * w[i] - on[i] * m2);
          hv[i] *= yn[i];
          fa[i] = dn * on[i];
          fm[i] = dg;
        }
        if (p.dx) store<T, V>(reinterpret_cast<T *>(p.dx) + r * p.ld_dx + c, dxv);
        if (p.dout) store<T, V>(reinterpret_cast<T *>(p.dout) + r * p.ld_do + c, dov);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (NV) {
            a_pre[j][i] += hv[i];
            a_post[j][i] += fa[i];
            a_gate[j][i] += fm[i];
          } else {
            ws_pre[c + i] += hv[i];
            ws_post[c + i] += fa[i];
            if (p.dgate) gate_sum[c + i] += fm[i];
          }
        }
      });
    }
    if (p.dgate)
      each([&](int j, int c) {
        float t[V];
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = NV ? a_gate[j][i] : gate_sum[c + i];
        if (p.split == 1) {  // this block saw all rows of the gate row
          float g[V];
          load<T, V>(gate + c, g);
#pragma unroll
          for (int i = 0; i < V; ++i) t[i] *= slope(p.act, g[i]);
          store<T, V>(reinterpret_cast<T *>(p.dgate) + gi * p.ld_dg + c, t);
        } else if (NV) {
#pragma unroll
          for (int i = 0; i < V; ++i) gate_sum[c + i] = t[i];
        }
      });
  }
  if (NV)
    each([&](int j, int c) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (p.dw_pre) ws_pre[c + i] = a_pre[j][i];
        if (p.dw_post) ws_post[c + i] = a_post[j][i];
      }
    });
}

// ---------------------------------------------------------------------------
// Staged kernels: rows in 16-byte vectors, at most 8192 columns.  A block walks
// work items (runs of rows that share a gate row) with 8 columns a thread,
// worked on as two quads so that 64 registers do and 1024 threads an SM hide
// the generator's and the reductions' latencies (16 columns a thread at 128
// registers: train 162, gradient 258 us).  A thread copies its own vectors of the
// next rows into its own shared memory (cp.async, a few rows deep), so no
// barrier guards the copies.  What a column needs for every row stays with its
// thread for the item's rows: the activated gate in registers, the weights in
// shared memory.
// ---------------------------------------------------------------------------
constexpr int STAGED_COLS = 8192;
constexpr int FWD_QUADS = 4, BWD_QUADS = 4;
constexpr int STAGED_SMEM = 220 * 1024;
// A gate row shared by this few rows is copied along with each of them.
constexpr int GATE_WITH_ROWS = 4;

// A block's rows in the order of its work items
struct Walk {
  int per_gate, per_item, row, end, item, items, split;
  __device__ Walk(int per_gate_, int per_item_, int gates, int split_)
      : per_gate(per_gate_), per_item(per_item_), item(blockIdx.x), items(gates * split_), split(split_) {
    open();
  }
  __device__ void open() {  // the item's rows; items without rows are passed over
    for (; item < items; item += gridDim.x) {
      const int g = item / split, first = g * per_gate;
      row = first + (item - g * split) * per_item;
      end = min(row + per_item, first + per_gate);
      if (row < end) return;
    }
  }
  __device__ bool live() const { return item < items; }
  __device__ void next() {
    if (++row < end) return;
    item += gridDim.x;
    open();
  }
};

// A thread's NQ quads of columns and its share of the row buffers.  16-bit
// types: quads 2j and 2j + 1 are vector j; fp32: quad k is vector k.  A thread's
// vectors are a block's width apart.
template <typename T, int NQ>
struct Mine {
  static constexpr int PER = sizeof(T) == 4 ? 1 : 2;  // quads of a vector
  static constexpr int NV = NQ / PER;
  int threads, arrays, ahead, turn;
  char *buf;
  __device__ Mine(char *smem, int arrays_, int ahead_)
      : threads(blockDim.x), arrays(arrays_), ahead(ahead_), turn(0), buf(smem + threadIdx.x * 16) {}
  // first column of vector j and of quad k
  __device__ __forceinline__ int vector(int j) const {
    return ((int)threadIdx.x + j * threads) * (16 / (int)sizeof(T));
  }
  __device__ __forceinline__ int quad(int k) const { return vector(k / PER) + 4 * (k % PER); }
  // vector j / quad k of `slot`, one of the 16-byte-per-thread planes
  __device__ __forceinline__ char *plane(int slot, int j) const { return buf + (size_t)(slot * NV + j) * threads * 16; }
  __device__ __forceinline__ char *plane_quad(int slot, int k) const {
    return plane(slot, k / PER) + 8 * (k % PER);
  }
  __device__ __forceinline__ char *row_vector(int a, int j) const { return plane(turn * arrays + a, j); }
  __device__ __forceinline__ char *row_quad(int a, int k) const { return plane_quad(turn * arrays + a, k); }
  __device__ __forceinline__ void next() { turn = turn + 1 == ahead ? 0 : turn + 1; }
  // the oldest row in flight has landed
  __device__ __forceinline__ void wait() const {
    if (ahead == 3) cp_async_wait<2>();
    else if (ahead == 2) cp_async_wait<1>();
    else cp_async_wait<0>();
  }
};
// Quads' results as whole 16-byte stores
template <typename T>
struct Writer {
  typename Quad<T>::Word first;
  __device__ __forceinline__ void put(int k, T *row, int col, const float (&f)[4]) {
    const typename Quad<T>::Word w = Quad<T>::put(f);
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<uint4 *>(row + col) = w;
    } else {
      if (k % 2 == 0) first = w;
      else *reinterpret_cast<uint4 *>(row + col - 4) = make_uint4(first.x, first.y, w.x, w.y);
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

template <typename T, int NQ>
__global__ void __launch_bounds__(NQ == 2 ? 1024 : 512) block_norm_staged_kernel(const Fwd p, int gate_with_rows, int ahead_rows) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float buf[2 * 32];
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  // x, o and, where it changes from row to row, the gate; then w_pre
  using M = Mine<T, NQ>;
  M my(smem, 2 + gate_with_rows, ahead_rows);
  const int w_slot = ahead_rows * my.arrays;
  const float inv = 1.f / p.cols;
  const T *w_post = reinterpret_cast<const T *>(p.w_post), *w_pre = reinterpret_cast<const T *>(p.w_pre);
  Walk ahead(p.per_gate, p.per_item, p.gates, p.split), now = ahead;
  auto fetch = [&]() {  // the next row, into the slot that is free
    if (ahead.live()) {
      const int r = ahead.row;
#pragma unroll
      for (int j = 0; j < M::NV; ++j) {
        const int c = my.vector(j);
        if (c < p.cols) {
          cp_async16(my.row_vector(0, j), at<T>(p.x, r, p.ldx) + c);
          if (p.o) cp_async16(my.row_vector(1, j), at<T>(p.o, r, p.ldo) + c);
          if (gate_with_rows)
            cp_async16(my.row_vector(2, j), at<T>(p.gate, ahead.item / p.split, p.ldg) + c);
        }
      }
      ahead.next();
    }
    cp_async_commit();
  };
  for (int i = 0; i < ahead_rows; ++i, my.next()) fetch();
  if (w_pre)
#pragma unroll
    for (int j = 0; j < M::NV; ++j)
      if (my.vector(j) < p.cols)
        *reinterpret_cast<uint4 *>(my.plane(w_slot, j)) = *reinterpret_cast<const uint4 *>(w_pre + my.vector(j));
  float factor[NQ][4];
  int half = 0, item = -1;
  for (; now.live(); now.next()) {
    const int r = now.row;
    if (p.o && (now.item != item) && !gate_with_rows) {
      item = now.item;
      const T *gate = p.gate ? at<T>(p.gate, item / p.split, p.ldg) : nullptr;
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        const int c = my.quad(k);
        if (c < p.cols) factor_of<T>(p.scale, p.act, gate ? gate + c : nullptr, w_post ? w_post + c : nullptr, factor[k]);
      }
    }
    my.wait();
    if (p.o && gate_with_rows)
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        const int c = my.quad(k);
        if (c < p.cols) factor_of<T>(p.scale, p.act, my.row_quad(2, k), w_post ? w_post + c : nullptr, factor[k]);
      }
    float rstd_o = 1.f;
    if (p.o && p.post_norm) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NQ; ++k)
        if (my.quad(k) < p.cols) {
          float ov[4];
          Quad<T>::get(my.row_quad(1, k), ov);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[0] += ov[i] * ov[i];
        }
      group_sums<1>(s, buf, warp, warps, half);
      rstd_o = rsqrtf(s[0] * inv + p.eps);
      if (threadIdx.x == 0 && p.rstd_post) p.rstd_post[r] = rstd_o;
    }
    float y[NQ][4], s[1] = {0.f};
    Writer<T> out;
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const int c = my.quad(k);
      if (c < p.cols) {
        Quad<T>::get(my.row_quad(0, k), y[k]);
        if (p.o) {
          float ov[4];
          Quad<T>::get(my.row_quad(1, k), ov);
          const float ks = p.drop ? rstd_o * p.rnd.keep_scale : rstd_o;
          uint32_t word[4] = {~0u, ~0u, ~0u, ~0u};
          if (p.drop) random_words(p.rnd, ((uint64_t)r * p.cols + c) >> 2, word);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (word[i] >= p.rnd.threshold) y[k][i] += ov[i] * ks * factor[k][i];
          out.put(k, at<T>(p.y, r, p.ldy), c, y[k]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[0] += y[k][i] * y[k][i];
      }
    }
    fetch();
    my.next();
    if (!p.h && !p.rstd_pre) continue;
    group_sums<1>(s, buf, warp, warps, half);
    const float rstd_y = rsqrtf(s[0] * inv + p.eps);
    if (threadIdx.x == 0 && p.rstd_pre) p.rstd_pre[r] = rstd_y;
    if (!p.h) continue;
#pragma unroll
    for (int k = 0; k < NQ; ++k)
      if (my.quad(k) < p.cols) {
        float w[4] = {1.f, 1.f, 1.f, 1.f};
        if (w_pre) Quad<T>::get(my.plane_quad(w_slot, k), w);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[k][i] *= rstd_y * w[i];
        out.put(k, at<T>(p.h, r, p.ldh), my.quad(k), y[k]);
      }
  }
}

// Backward.  Per column the block keeps two sums: of dh yn (dw_pre), and over
// an item's rows S = sum drop dx on, from which both dw_post = sum over gates
// of scale act S and dgate = scale act' w_post S follow.
template <typename T, int NQ>
__global__ void __launch_bounds__(NQ == 2 ? 1024 : 512) block_norm_bwd_staged_kernel(const Bwd p, int gate_with_rows, int ahead_rows) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float buf[2 * 32 * 3];
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32;
  // dy, dh, y, o and, where it changes from row to row, the gate; then w_pre,
  // then this thread's columns of dw_post, summed over the items
  using M = Mine<T, NQ>;
  M my(smem, 4 + gate_with_rows, ahead_rows);
  const int w_slot = ahead_rows * my.arrays;
  float *post = reinterpret_cast<float *>(smem + (size_t)(w_slot + 1) * M::NV * blockDim.x * 16) + threadIdx.x;
  const float inv = 1.f / p.cols;
  const T *w_post = reinterpret_cast<const T *>(p.w_post), *w_pre = reinterpret_cast<const T *>(p.w_pre);
  Walk ahead(p.per_gate, p.per_item, p.gates, p.split), now = ahead;
  auto fetch = [&]() {  // the next row, into the slot that is free
    if (ahead.live()) {
      const int r = ahead.row;
#pragma unroll
      for (int j = 0; j < M::NV; ++j) {
        const int c = my.vector(j);
        if (c < p.cols) {
          if (p.dy) cp_async16(my.row_vector(0, j), at<T>(p.dy, r, p.ld_dy) + c);
          if (p.dh) {
            cp_async16(my.row_vector(1, j), at<T>(p.dh, r, p.ld_dh) + c);
            cp_async16(my.row_vector(2, j), at<T>(p.y, r, p.ldy) + c);
          }
          if (p.o) cp_async16(my.row_vector(3, j), at<T>(p.o, r, p.ldo) + c);
          if (gate_with_rows)
            cp_async16(my.row_vector(4, j), at<T>(p.gate, ahead.item / p.split, p.ldg) + c);
        }
      }
      ahead.next();
    }
    cp_async_commit();
  };
  for (int i = 0; i < ahead_rows; ++i, my.next()) fetch();
  if (w_pre)
#pragma unroll
    for (int j = 0; j < M::NV; ++j)
      if (my.vector(j) < p.cols)
        *reinterpret_cast<uint4 *>(my.plane(w_slot, j)) = *reinterpret_cast<const uint4 *>(w_pre + my.vector(j));
  float factor[NQ][4], a_pre[NQ][4], a_s[NQ][4];
#pragma unroll
  for (int k = 0; k < NQ; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      factor[k][i] = a_pre[k][i] = a_s[k][i] = 0.f;
      post[(k * 4 + i) * blockDim.x] = 0.f;
    }
  auto gate_row = [&](int item) {
    return p.gate ? at<T>(p.gate, item / p.split, p.ldg) : nullptr;
  };
  // an item's S goes to dw_post's sums and to the gate's gradient (directly
  // where the item is all of the gate row's rows)
  auto flush = [&](int item) {
    if (!p.o || item < 0) return;
    const T *gate = gate_row(item);
    Writer<T> out;
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const int c = my.quad(k);
      if (c < p.cols) {
        float g[4], w[4] = {1.f, 1.f, 1.f, 1.f}, d[4];
        if (gate) Quad<T>::get(gate + c, g);
        if (w_post) Quad<T>::get(w_post + c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = p.scale * a_s[k][i];
          post[(k * 4 + i) * blockDim.x] += gate ? activate(p.act, g[i]) * s : s;
          d[i] = s * w[i];
          a_s[k][i] = 0.f;
        }
        if (!p.dgate) continue;
        if (p.split == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] *= slope(p.act, g[i]);
          out.put(k, at<T>(p.dgate, item, p.ld_dg), c, d);
        } else {
          float *sums = p.ws + 2 * (int64_t)gridDim.x * p.cols + (int64_t)item * p.cols;
          *reinterpret_cast<float4 *>(sums + c) = make_float4(d[0], d[1], d[2], d[3]);
        }
      }
    }
  };
  // yn, dx without its mean term and dh of a quad; s0 += dh w_pre yn
  auto front = [&](int k, float ry, float (&yn)[4], float (&g0)[4], float (&hv)[4], float &s0) {
    float w[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) yn[i] = g0[i] = hv[i] = 0.f;
    if (p.dy) Quad<T>::get(my.row_quad(0, k), g0);
    if (!p.dh) return;
    Quad<T>::get(my.row_quad(1, k), hv);
    Quad<T>::get(my.row_quad(2, k), yn);
    if (w_pre) Quad<T>::get(my.plane_quad(w_slot, k), w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      yn[i] *= ry;
      const float t = hv[i] * w[i];
      g0[i] += ry * t;
      s0 += t * yn[i];
    }
  };
  int half = 0, item = -1;
  for (; now.live(); now.next()) {
    const int r = now.row;
    const float ry = p.dh ? p.rstd_pre[r] : 0.f;
    const float ro = p.o && p.post_norm ? p.rstd_post[r] : 1.f;
    if (now.item != item) {
      flush(item);
      item = now.item;
      const T *gate = gate_row(item);
      if (p.o && !gate_with_rows)
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
          const int c = my.quad(k);
          if (c < p.cols) factor_of<T>(p.scale, p.act, gate ? gate + c : nullptr, w_post ? w_post + c : nullptr, factor[k]);
        }
    }
    my.wait();
    uint32_t kept = 0u;  // bit 4k + i: element i of quad k is kept
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const int c = my.quad(k);
      if (c < p.cols) {
        if (p.o && gate_with_rows)
          factor_of<T>(p.scale, p.act, my.row_quad(4, k), w_post ? w_post + c : nullptr, factor[k]);
        uint32_t word[4] = {~0u, ~0u, ~0u, ~0u};
        if (p.o && p.drop) random_words(p.rnd, ((uint64_t)r * p.cols + c) >> 2, word);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (word[i] >= p.rnd.threshold) kept |= 1u << (4 * k + i);
        float yn[4], g0[4], hv[4];
        front(k, ry, yn, g0, hv, s[0]);
        if (p.o && p.post_norm) {
          float ov[4];
          Quad<T>::get(my.row_quad(3, k), ov);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float q = word[i] >= p.rnd.threshold ? factor[k][i] * ov[i] : 0.f;
            s[1] += g0[i] * q;
            s[2] += yn[i] * q;
          }
        }
      }
    }
    group_sums<3>(s, buf, warp, warps, half);
    const float m1 = ry * s[0] * inv;  // dx = g0 - yn * m1
    const float ks = p.drop ? p.rnd.keep_scale : 1.f;
    const float m2 = p.post_norm ? ks * ro * (s[1] - m1 * s[2]) * inv : 0.f;  // mean(dn w_post on)
    Writer<T> out_x, out_o;
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const int c = my.quad(k);
      if (c < p.cols) {
        float yn[4], g0[4], hv[4], unused = 0.f;
        front(k, ry, yn, g0, hv, unused);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a_pre[k][i] += hv[i] * yn[i];
          g0[i] -= yn[i] * m1;  // dx
        }
        if (p.dx) out_x.put(k, at<T>(p.dx, r, p.ld_dx), c, g0);
        if (p.o) {
          float ov[4];
          Quad<T>::get(my.row_quad(3, k), ov);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float on = ov[i] * ro;
            // a dropped element passes nothing on, whatever its values
            const float d = (kept >> (4 * k + i)) & 1u ? g0[i] * ks : 0.f;
            a_s[k][i] += d * on;
            ov[i] = ro * (d * factor[k][i] - on * m2);
          }
          if (p.dout) out_o.put(k, at<T>(p.dout, r, p.ld_do), c, ov);
        }
      }
    }
    fetch();
    my.next();
  }
  flush(item);
#pragma unroll
  for (int k = 0; k < NQ; ++k) {
    const int c = my.quad(k);
    if (c < p.cols) {
      if (p.dw_pre)
        *reinterpret_cast<float4 *>(p.ws + (int64_t)blockIdx.x * p.cols + c) =
            make_float4(a_pre[k][0], a_pre[k][1], a_pre[k][2], a_pre[k][3]);
      if (p.dw_post)
        *reinterpret_cast<float4 *>(p.ws + ((int64_t)gridDim.x + blockIdx.x) * p.cols + c) =
            make_float4(post[(k * 4) * blockDim.x], post[(k * 4 + 1) * blockDim.x], post[(k * 4 + 2) * blockDim.x],
                        post[(k * 4 + 3) * blockDim.x]);
    }
  }
}

// Column sums of the partials: y 0 dw_pre, 1 dw_post, 2 + g the gate rows.
// A block adds 32 columns: warp w takes partials w, w + 8, ..., then the eight
// sums are added in order.
template <typename T>
__global__ void __launch_bounds__(256) sum_partials_kernel(const Bwd p, int blocks) {
  __shared__ float part[8][33];
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
  if (c < p.cols)
    for (int i = w; i < n; i += 8) s += from[(int64_t)i * p.cols + c];
  part[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w != 0 || c >= p.cols) return;
  s = 0.f;
  for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
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
// Threads of a row for rows of `cols` elements in vectors of V: whole warps,
// at most `most`, each with at most `nv` vectors (0: the row does not fit)
static int threads_of(int cols, int V, int nv, int most) {
  const int vecs = (cols + V - 1) / V;
  const int t = ((vecs + nv - 1) / nv + 31) / 32 * 32;
  return t <= most ? t : 0;
}

// Resident blocks of a staged kernel: 1024 threads an SM at 2 quads, 512 or 768 at 4
static int staged_per_sm(int threads, int nq) { return std::max(1, (nq == 2 ? 1024 : 512) / threads); }
static int64_t staged_blocks(int64_t rows, int threads, int nq, int num_sms) {
  return std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms * staged_per_sm(threads, nq)));
}
// Rows to copy ahead: up to three, as many as leave room for `blocks` blocks an SM
static int ahead_of(size_t arrays, size_t fixed, size_t vectors, int blocks) {
  const size_t room = STAGED_SMEM / std::max(1, blocks) / vectors;
  return room < fixed + 2 * arrays ? 1 : room < fixed + 3 * arrays ? 2 : 3;
}
// Split of a gate row's rows so that all items together give every block one
static int64_t split_of(int64_t gates, int64_t per_gate, int64_t blocks) {
  if (gates >= blocks) return 1;
  return std::max<int64_t>(1, std::min<int64_t>(per_gate, blocks / gates));
}
// Quads of a thread's columns, and the threads of a staged block
static int staged_quads(int cols, int quads) { return cols <= 2048 ? 2 : quads; }
static int staged_threads(int cols, int nq) { return (cols / 4 + 32 * nq - 1) / (32 * nq) * 32; }

template <typename T, int V, int NV>
static cudaError_t run_fwd(const Fwd &p, int tpr, int num_sms, cudaStream_t st) {
  const int rpb = std::max(1, 128 / tpr);
  const int64_t blocks = std::min<int64_t>((p.rows + rpb - 1) / rpb, (int64_t)num_sms * 64);
  block_norm_kernel<T, V, NV><<<(unsigned)blocks, dim3(tpr, rpb), rpb * 64 * sizeof(float), st>>>(p);
  return cudaGetLastError();
}
template <typename T, int V>
static cudaError_t fwd(Fwd p, int num_sms, cudaStream_t st) {
  if constexpr (V > 1) {
    if (p.cols <= STAGED_COLS) {
      const int nq = staged_quads(p.cols, FWD_QUADS), threads = staged_threads(p.cols, nq);
      const int64_t most = staged_blocks(p.rows, threads, nq, num_sms);
      p.split = (int)split_of(p.gates, p.per_gate, most);
      p.per_item = (p.per_gate + p.split - 1) / p.split;
      const int blocks = (int)std::min<int64_t>(most, (int64_t)p.gates * p.split);
      const int with_rows = p.gate && p.per_gate <= GATE_WITH_ROWS;
      const size_t vectors = 4 * nq * sizeof(T) * threads;  // a row's bytes of one array
      const int ahead = ahead_of(2 + with_rows, 1, vectors, staged_per_sm(threads, nq));
      const size_t smem = ((size_t)ahead * (2 + with_rows) + 1) * vectors;
      auto kern = nq == 2 ? block_norm_staged_kernel<T, 2> : block_norm_staged_kernel<T, FWD_QUADS>;
      const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (err != cudaSuccess) return err;
      kern<<<blocks, threads, smem, st>>>(p, with_rows, ahead);
      return cudaGetLastError();
    }
    if (const int t = threads_of(p.cols, V, 2, 1024)) return run_fwd<T, V, 2>(p, t, num_sms, st);
  } else {
    // single elements: 4 or 8 a thread
    if (const int t = threads_of(p.cols, 1, 4, 256)) return run_fwd<T, 1, 4>(p, t, num_sms, st);
    if (const int t = threads_of(p.cols, 1, 8, 1024)) return run_fwd<T, 1, 8>(p, t, num_sms, st);
  }
  return run_fwd<T, V, 0>(p, 1024, num_sms, st);
}

// The backward's launch: threads and blocks for rows in vectors of V
struct BwdPlan {
  bool staged;
  int threads, nv;  // a thread's quads, or the plain kernel's vectors in registers (0: none)
  int64_t blocks;
};
static BwdPlan plan_bwd(int64_t rows, int cols, int V, int num_sms) {
  if (V > 1 && cols <= STAGED_COLS) {
    const int nq = staged_quads(cols, BWD_QUADS), t = staged_threads(cols, nq);
    return BwdPlan{true, t, nq, staged_blocks(rows, t, nq, num_sms)};
  }
  const int n = V == 1 ? 8 : 0;
  const int t = n ? threads_of(cols, V, n, 512) : 0;
  const int threads = t ? t : 512;
  return BwdPlan{false, threads, t ? n : 0,
                 std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms * std::max(1, 1024 / threads)))};
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
      const int with_rows = p.gate && p.per_gate <= GATE_WITH_ROWS;
      const size_t vectors = 4 * plan.nv * sizeof(T) * plan.threads;
      const size_t sums = sizeof(float) / sizeof(T);  // dw_post's sums, in rows
      const int ahead = ahead_of(4 + with_rows, 1 + sums, vectors, staged_per_sm(plan.threads, plan.nv));
      const size_t smem = ((size_t)ahead * (4 + with_rows) + 1 + sums) * vectors;
      auto kern = plan.nv == 2 ? block_norm_bwd_staged_kernel<T, 2> : block_norm_bwd_staged_kernel<T, BWD_QUADS>;
      err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (err != cudaSuccess) return err;
      kern<<<blocks, plan.threads, smem, st>>>(p, with_rows, ahead);
    } else {
      block_norm_bwd_kernel<T, V, 0><<<blocks, plan.threads, 0, st>>>(p);
    }
  } else {
    if (plan.nv) block_norm_bwd_kernel<T, 1, 8><<<blocks, plan.threads, 0, st>>>(p);
    else block_norm_bwd_kernel<T, 1, 0><<<blocks, plan.threads, 0, st>>>(p);
  }
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const bool gates = p.dgate && p.split > 1;
  if (p.dw_pre || p.dw_post || gates)
    err = launch_pdl(sum_partials_kernel<T>, dim3((p.cols + 31) / 32, 2 + (gates ? p.gates : 0)), dim3(256), 0, st, p,
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
    const int64_t items = gates && (split > 1 || (!plan.staged && plan.nv == 0)) ? gates * split : 0;
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
  p.cols = a.cols, p.act = a.gate_act, p.post_norm = !(a.flags & SYM_NORM_NO_POST);
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
  const bool vec = vec_ok({p.dy, p.dh, p.dh ? p.y : nullptr, p.o, p.w_post, p.w_pre, p.gate, p.dx, p.dout, p.dgate},
                          {p.dy ? p.ld_dy : 0, p.dh ? p.ld_dh : 0, p.dh ? p.ldy : 0, p.o ? p.ldo : 0,
                           p.gate ? p.ldg : 0, p.dx ? p.ld_dx : 0, p.dout ? p.ld_do : 0, p.dgate ? p.ld_dg : 0},
                          p.cols, es);
  if (a.dtype == SYM_BF16) return vec ? bwd<__nv_bfloat16, 8>(p, num_sms, st) : bwd<__nv_bfloat16, 1>(p, num_sms, st);
  if (a.dtype == SYM_FP16) return vec ? bwd<__half, 8>(p, num_sms, st) : bwd<__half, 1>(p, num_sms, st);
  return vec ? bwd<float, 4>(p, num_sms, st) : bwd<float, 1>(p, num_sms, st);
}

}  // namespace symmoe
