// rows_ops.cu -- row-wise operators between and after the grouped products:
// SwiGLU of expert rows with the row's routing weight, forward and backward,
// and dropout whose mask is recomputed from a counter instead of stored.
//
//   h  = rw * silu(g) * u            silu(g) = g * s, s = 1 / (1 + exp(-g))
//   dg = rw * dh * u * s * (1 + g * (1 - s)),  du = rw * dh * silu(g),
//   d_rw = sum over the row of dh * silu(g) * u
//   y  = residual + x * [word(i) >= p * 2^32] / (1 - p)
//
// All are bound by their bytes.  A row is walked in 16-byte vectors; where the
// rows start off a 16-byte boundary (odd row lengths) all tensors of a call
// are off by the same amount, and only the vectors cut by the row's ends are
// moved element by element.  Measured (bf16, copy rate 6.69 TB/s): forward 65536 x
// 2048 133 us (6.0 TB/s), backward 32768 x 14336 819 us (5.7 TB/s), dropout with
// residual 16384 x 4096 67 us (6.0 TB/s).
#include <algorithm>

#include "rows_dev.cuh"

namespace symmoe {
namespace rows {

constexpr int THREADS = 256;

struct View {
  char *ptr;
  int64_t ld, slot;  // bytes
};

struct RowArgs {
  View a, b, c, d, e;  // swiglu: g u h; backward: g u dh dg du; dropout: x residual y
  const float *rw;
  float *drw;
  int64_t rw_slot, drw_slot;
  const int32_t *total;
  int64_t total_slot;
  int64_t rows;
  int slots, cols;
};

template <typename T>
__device__ __forceinline__ T *row_of(const View &v, int d, int64_t r) {
  return reinterpret_cast<T *>(v.ptr + d * v.slot + r * v.ld);
}
// elements between the 16-byte boundary at or before p and p (V = 1: none)
template <typename T, int V>
__device__ __forceinline__ int skew(const T *p) {
  return V == 1 ? 0 : (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// rows a slot holds: total[slot] where given (values outside [0, rows] are cut)
__device__ __forceinline__ int64_t live_rows(const RowArgs &p, int d) {
  if (!p.total) return p.rows;
  const int64_t t = p.total[d * p.total_slot];
  return t < 0 ? 0 : t > p.rows ? p.rows : t;
}

// (1 + exp(-g) may overflow: the quotient is then 0, the limit)
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// blockDim (threads of a row, rows of a block); grid (blocks, slots)
template <typename T, int V>
__global__ void __launch_bounds__(THREADS) swiglu_kernel(const RowArgs p) {
  const int d = blockIdx.y;
  const int64_t rows = live_rows(p, d);
  for (int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; r < rows; r += (int64_t)gridDim.x * blockDim.y) {
    const T *g = row_of<T>(p.a, d, r), *u = row_of<T>(p.b, d, r);
    T *h = row_of<T>(p.c, d, r);
    const float w = p.rw ? p.rw[d * p.rw_slot + r] : 1.f;
    for (int c = (int)threadIdx.x * V - skew<T, V>(g); c < p.cols; c += blockDim.x * V) {
      float gv[V], uv[V];
      load_part<T, V>(g, c, p.cols, gv);
      load_part<T, V>(u, c, p.cols, uv);
#pragma unroll
      for (int i = 0; i < V; ++i) gv[i] = w * (gv[i] * sigmoid(gv[i])) * uv[i];
      store_part<T, V>(h, c, p.cols, gv);
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS, 6) swiglu_bwd_kernel(const RowArgs p) {
  __shared__ float buf[2][32];
  const int d = blockIdx.y;
  const int64_t rows = live_rows(p, d);
  const int warps_row = blockDim.x / 32, warp = threadIdx.x / 32, base = threadIdx.y * warps_row;
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < rows; r0 += step) {
    const int64_t r = r0 + threadIdx.y;
    float sum = 0.f;
    if (r < rows) {
      const T *g = row_of<T>(p.a, d, r), *u = row_of<T>(p.b, d, r), *dh = row_of<T>(p.c, d, r);
      T *dg = row_of<T>(p.d, d, r), *du = row_of<T>(p.e, d, r);
      const float w = p.rw ? p.rw[d * p.rw_slot + r] : 1.f;
      for (int c = (int)threadIdx.x * V - skew<T, V>(g); c < p.cols; c += blockDim.x * V) {
        float gv[V], uv[V], hv[V];
        load_part<T, V>(g, c, p.cols, gv);
        load_part<T, V>(u, c, p.cols, uv);
        load_part<T, V>(dh, c, p.cols, hv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float s = sigmoid(gv[i]), silu = gv[i] * s, wh = w * hv[i];
          sum += hv[i] * silu * uv[i];
          gv[i] = wh * uv[i] * (s * (1.f + gv[i] * (1.f - s)));
          uv[i] = wh * silu;
        }
        store_part<T, V>(dg, c, p.cols, gv);
        store_part<T, V>(du, c, p.cols, uv);
      }
    }
    if (!p.drw) continue;
    float v[1] = {sum};
    warp_sums<1>(v);
    if (warps_row > 1) {
      if ((threadIdx.x & 31) == 0) buf[turn][base + warp] = v[0];
      __syncthreads();
      if (threadIdx.x == 0) {
        v[0] = 0.f;
        for (int i = 0; i < warps_row; ++i) v[0] += buf[turn][base + i];
      }
      turn ^= 1;
    }
    if (threadIdx.x == 0 && r < rows) p.drw[d * p.drw_slot + r] = v[0];
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS) dropout_kernel(const RowArgs p, const Random rnd) {
  const int d = blockIdx.y;
  for (int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; r < p.rows; r += (int64_t)gridDim.x * blockDim.y) {
    const T *x = row_of<T>(p.a, d, r);
    T *y = row_of<T>(p.c, d, r);
    const uint64_t first = ((uint64_t)d * p.rows + r) * p.cols;  // index of the row's first element
    for (int64_t c = (int64_t)threadIdx.x * V - skew<T, V>(x); c < p.cols; c += blockDim.x * V) {
      float xv[V], k[V];
      load_part<T, V>(x, (int)c, p.cols, xv);
      keep_factors<V>(rnd, first + c, k);
      if (p.b.ptr) {
        float rv[V];
        load_part<T, V>(row_of<T>(p.b, d, r), (int)c, p.cols, rv);
#pragma unroll
        for (int i = 0; i < V; ++i) xv[i] = k[i] != 0.f ? rv[i] + xv[i] * k[i] : rv[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) xv[i] = k[i] != 0.f ? xv[i] * k[i] : 0.f;
      }
      store_part<T, V>(y, (int)c, p.cols, xv);
    }
  }
}

// The same over one run of n contiguous elements (element i is number i of the
// stream): no rows to address.  Eight elements a thread at a time, their two
// blocks of words side by side, and many warps: 66 us at 16384 x 4096 (bf16,
// residual; 6.1 TB/s), against 71 and 76 with 16 and 32 elements.
template <typename T>
__global__ void __launch_bounds__(THREADS) dropout_flat_kernel(const T *x, const T *res, T *y, int64_t n,
                                                               const Random rnd) {
  constexpr int V = Elem<T>::VEC, U = 8 / V;
  const int64_t vecs = n / V, step = (int64_t)gridDim.x * THREADS;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < vecs; i += U * step) {
    uint4 a[U], b[U];
    uint64_t block[2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = i + u * step;
      b[u] = make_uint4(0, 0, 0, 0);
      if (at < vecs) {
        a[u] = reinterpret_cast<const uint4 *>(x)[at];
        if (res) b[u] = reinterpret_cast<const uint4 *>(res)[at];
      }
#pragma unroll
      for (int q = 0; q < V / 4; ++q) block[u * (V / 4) + q] = (uint64_t)at * (V / 4) + q;
    }
    const uint32_t kept = kept_bits<2>(rnd, block);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u * step >= vecs) continue;
      float f[V], r[V];
      unpack<T, V>(a[u], f);
      unpack<T, V>(b[u], r);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if ((kept >> (u * V + j)) & 1u) r[j] += f[j] * rnd.keep_scale;
      reinterpret_cast<uint4 *>(y)[i + u * step] = pack<T, V>(r);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < n % V) {
    const int64_t at = vecs * V + threadIdx.x;
    uint32_t word[4];
    random_words(rnd, (uint64_t)at >> 2, word);
    const bool kept = word[at & 3] >= rnd.threshold;
    const float r = res ? Elem<T>::get(res[at]) : 0.f;
    y[at] = Elem<T>::put(kept ? r + Elem<T>::get(x[at]) * rnd.keep_scale : r);
  }
}

static View view_of(const sym_rows *r, int64_t es) {
  if (!r) return View{nullptr, 0, 0};
  return View{reinterpret_cast<char *>(r->ptr), r->ld * es, r->slots > 1 ? r->slot_stride * es : 0};
}

struct Shape {
  dim3 grid, block;
};
// Threads of a row: enough for one vector each up to a block of 256, in powers
// of two from a warp on; the block's other threads take further rows.
// At most `per_sm` blocks an SM: a forward row is little work (prefill shape, 32
// blocks 134 us, a block a row 139); the backward with its five streams runs
// better as many short blocks (32768 x 14336: 32 blocks 901 us, a block a row
// 819 with six resident; at their 40 registers the 16-bit forms spill, 72 bytes
// stored and 60 loaded a thread).
static Shape shape_of(int64_t rows, int slots, int cols, int vec, int num_sms, int per_sm = 32) {
  int tpr = 32;
  while (tpr < THREADS && tpr * vec < cols) tpr *= 2;
  const int rpb = THREADS / tpr;
  const int64_t blocks = std::min<int64_t>((rows + rpb - 1) / rpb, (int64_t)num_sms * per_sm);
  return Shape{dim3((unsigned)std::max<int64_t>(1, blocks), slots), dim3(tpr, rpb)};
}

// Do all tensors of a call start their rows at the same place of a 16-byte
// line, so that they can be walked in the same vectors?
static bool same_skew(std::initializer_list<const sym_rows *> all, int64_t es) {
  const sym_rows *f = *all.begin();
  for (const sym_rows *r : all) {
    if (!r) continue;
    if ((r->ptr - f->ptr) % 16 || ((r->ld - f->ld) * es) % 16 ||
        (r->slots > 1 && ((r->slot_stride - f->slot_stride) * es) % 16))
      return false;
  }
  return true;
}

}  // namespace rows

#define SYM_ROWS_LAUNCH(KERNEL, ...)                                                                      \
  switch (dtype) {                                                                                        \
    case SYM_BF16:                                                                                        \
      if (vec) rows::KERNEL<__nv_bfloat16, 8><<<s.grid, s.block, 0, st>>>(__VA_ARGS__);                   \
      else rows::KERNEL<__nv_bfloat16, 1><<<s.grid, s.block, 0, st>>>(__VA_ARGS__);                       \
      break;                                                                                              \
    case SYM_FP16:                                                                                        \
      if (vec) rows::KERNEL<__half, 8><<<s.grid, s.block, 0, st>>>(__VA_ARGS__);                          \
      else rows::KERNEL<__half, 1><<<s.grid, s.block, 0, st>>>(__VA_ARGS__);                              \
      break;                                                                                              \
    default:                                                                                              \
      if (vec) rows::KERNEL<float, 4><<<s.grid, s.block, 0, st>>>(__VA_ARGS__);                           \
      else rows::KERNEL<float, 1><<<s.grid, s.block, 0, st>>>(__VA_ARGS__);                               \
  }                                                                                                       \
  return cudaGetLastError();

static int64_t elem_size(int dtype) { return dtype == SYM_FP32 ? 4 : 2; }

cudaError_t launch_swiglu_rows(int dtype, const sym_rows &g, const sym_rows &u, const sym_rows &h, const float *rw,
                               int64_t rw_slot, const int32_t *total, int64_t total_slot, int num_sms,
                               cudaStream_t st) {
  using namespace rows;
  const int64_t es = elem_size(dtype);
  const bool vec = same_skew({&g, &u, &h}, es);
  RowArgs a = {};
  a.a = view_of(&g, es), a.b = view_of(&u, es), a.c = view_of(&h, es);
  a.rw = rw, a.rw_slot = rw_slot, a.total = total, a.total_slot = total_slot;
  a.rows = g.rows, a.slots = g.slots, a.cols = g.cols;
  const Shape s = shape_of(g.rows, g.slots, g.cols, vec ? (int)(16 / es) : 1, num_sms);
  SYM_ROWS_LAUNCH(swiglu_kernel, a)
}

cudaError_t launch_swiglu_rows_bwd(int dtype, const sym_rows &g, const sym_rows &u, const sym_rows &dh,
                                   const sym_rows &dg, const sym_rows &du, const float *rw, int64_t rw_slot,
                                   float *drw, int64_t drw_slot, const int32_t *total, int64_t total_slot,
                                   int num_sms, cudaStream_t st) {
  using namespace rows;
  const int64_t es = elem_size(dtype);
  const bool vec = same_skew({&g, &u, &dh, &dg, &du}, es);
  RowArgs a = {};
  a.a = view_of(&g, es), a.b = view_of(&u, es), a.c = view_of(&dh, es), a.d = view_of(&dg, es), a.e = view_of(&du, es);
  a.rw = rw, a.rw_slot = rw_slot, a.drw = drw, a.drw_slot = drw_slot, a.total = total, a.total_slot = total_slot;
  a.rows = g.rows, a.slots = g.slots, a.cols = g.cols;
  const Shape s = shape_of(g.rows, g.slots, g.cols, vec ? (int)(16 / es) : 1, num_sms, 4096);
  SYM_ROWS_LAUNCH(swiglu_bwd_kernel, a)
}

cudaError_t launch_dropout(int dtype, const sym_rows &x, const sym_rows *res, const sym_rows &y, uint64_t seed,
                           uint64_t offset, double drop, int num_sms, cudaStream_t st) {
  using namespace rows;
  const int64_t es = elem_size(dtype);
  const bool vec = same_skew({&x, &y, res}, es);
  const Random rnd = make_random(seed, offset, drop);
  RowArgs a = {};
  a.a = view_of(&x, es), a.b = view_of(res, es), a.c = view_of(&y, es);
  a.rows = x.rows, a.slots = x.slots, a.cols = x.cols;
  // rows that follow each other without gaps, on 16-byte boundaries: one run
  auto run = [&](const sym_rows *r) {
    return !r || (r->ptr % 16 == 0 && (r->rows == 1 || r->ld == r->cols) &&
                  (r->slots == 1 || r->slot_stride == r->rows * r->cols));
  };
  if (run(&x) && run(&y) && run(res)) {
    const int64_t n = x.rows * x.slots * x.cols, per = THREADS * 8;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + per - 1) / per, (int64_t)num_sms * 32);
    auto go = [&](auto zero) {
      using T = decltype(zero);
      dropout_flat_kernel<T><<<blocks, THREADS, 0, st>>>(reinterpret_cast<const T *>(x.ptr),
                                                         res ? reinterpret_cast<const T *>(res->ptr) : nullptr,
                                                         reinterpret_cast<T *>(y.ptr), n, rnd);
    };
    if (dtype == SYM_BF16) go(__nv_bfloat16{});
    else if (dtype == SYM_FP16) go(__half{});
    else go(float{});
    return cudaGetLastError();
  }
  const Shape s = shape_of(x.rows, x.slots, x.cols, vec ? (int)(16 / es) : 1, num_sms);
  SYM_ROWS_LAUNCH(dropout_kernel, a, rnd)
}

}  // namespace symmoe
