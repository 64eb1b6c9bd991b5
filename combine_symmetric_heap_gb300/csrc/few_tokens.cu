// few_tokens.cu -- a whole MoE layer for a few tokens: routing, the chosen experts'
// SwiGLU and the weighted sum, without a heap.
//
//   l = x Wr^T (or given); idx, w = top-k and softmax over it
//   h = silu(x Wg^T) * (x Wu^T);  out[t] = sum_j w[t][j] h[t, j] Wd^T
//
// Bound by the read of the chosen experts' weights.
#include <algorithm>

#include "rows_dev.cuh"

namespace symmoe {
namespace few_tokens {

using namespace rows;

struct Args {
  const uint16_t *x, *wg, *wu, *wd, *wr;
  float *logits;
  int32_t *idx;
  float *w;
  uint16_t *out;
  float *h;
  int64_t ldx, ld_out, g_group, g_ld, u_group, u_ld, d_group, d_ld, r_ld;
  int T, H, I, E, k;
};

template <typename T>
__device__ __forceinline__ float one(uint16_t v) {
  return Elem<T>::get(*reinterpret_cast<const T *>(&v));
}
template <typename T>
__device__ __forceinline__ float dot(const uint16_t *a, const uint16_t *b, int n) {
  float s[1] = {0.f};
  for (int c = (threadIdx.x & 31) * 8; c < n; c += 256) {
    float u[8], v[8];
    unpack<T, 8>(*reinterpret_cast<const uint4 *>(a + c), u);
    unpack<T, 8>(*reinterpret_cast<const uint4 *>(b + c), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += u[i] * v[i];
  }
  warp_sums<1>(s);
  return s[0];
}
__device__ __forceinline__ int64_t warp_index() { return (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; }

template <typename T>
__global__ void __launch_bounds__(256) router_kernel(const Args p) {
  const int64_t i = warp_index();
  if (i >= (int64_t)p.T * p.E) return;
  const int t = i / p.E, e = i % p.E;
  const float s = dot<T>(p.x + t * p.ldx, p.wr + e * p.r_ld, p.H);
  if ((threadIdx.x & 31) == 0) p.logits[i] = s;
}

__device__ __forceinline__ bool before(float a, int i, float b, int j) {  // does (a, i) rank before (b, j)?
  const bool na = a != a, nb = b != b;
  if (na != nb) return nb;
  if (!na && a != b) return a > b;
  return i < j;
}
// One warp a token: k rounds of the best expert left.
__global__ void __launch_bounds__(32) route_kernel(const Args p) {
  const int t = blockIdx.x, lane = threadIdx.x;
  const float *l = p.logits + (int64_t)t * p.E;
  float last = 0.f, mine = 0.f;
  int last_e = -1, my_e = 0;
  for (int j = 0; j < p.k; ++j) {
    float bv = 0.f;
    int be = -1;
    for (int e = lane; e < p.E; e += 32) {
      const float v = l[e];
      if (last_e >= 0 && !before(last, last_e, v, e)) continue;  // taken
      if (be < 0 || before(v, e, bv, be)) bv = v, be = e;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, bv, s);
      const int oe = __shfl_xor_sync(0xffffffffu, be, s);
      if (oe >= 0 && (be < 0 || before(ov, oe, bv, be))) bv = ov, be = oe;
    }
    last = bv, last_e = be;
    if (lane == j) mine = bv, my_e = be;
  }
  const float top = __shfl_sync(0xffffffffu, mine, 0);
  float z[1] = {lane < p.k && mine != -INFINITY ? expf(mine - top) : 0.f};
  const float e = z[0];
  warp_sums<1>(z);
  if (lane < p.k) {
    p.idx[t * p.k + lane] = my_e;
    p.w[t * p.k + lane] = e == 0.f ? 0.f : e / z[0];
  }
}

template <typename T>
__global__ void __launch_bounds__(256) up_kernel(const Args p) {
  const int64_t i = warp_index();
  if (i >= (int64_t)p.T * p.k * p.I) return;
  const int pair = i / p.I, f = i % p.I, e = p.idx[pair];
  if (p.logits[(int64_t)(pair / p.k) * p.E + e] == -INFINITY) return;
  const uint16_t *x = p.x + (pair / p.k) * p.ldx;
  const float g = dot<T>(x, p.wg + e * p.g_group + f * p.g_ld, p.H), u = dot<T>(x, p.wu + e * p.u_group + f * p.u_ld, p.H);
  if ((threadIdx.x & 31) == 0) p.h[i] = g / (1.f + __expf(-g)) * u;
}

template <typename T>
__global__ void __launch_bounds__(256) down_kernel(const Args p) {
  const int64_t i = warp_index();
  if (i >= (int64_t)p.T * p.H) return;
  const int t = i / p.H, f = i % p.H, lane = threadIdx.x & 31;
  float out = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int pair = t * p.k + j, e = p.idx[pair];
    if (p.logits[(int64_t)t * p.E + e] == -INFINITY) continue;
    const uint16_t *w = p.wd + e * p.d_group + f * p.d_ld;
    float s[1] = {0.f};
    for (int c = lane; c < p.I; c += 32) s[0] += p.h[(int64_t)pair * p.I + c] * one<T>(w[c]);
    warp_sums<1>(s);
    out += p.w[pair] * s[0];
  }
  const T v = Elem<T>::put(out);
  if (lane == 0) p.out[t * p.ld_out + f] = *reinterpret_cast<const uint16_t *>(&v);
}

template <typename T>
static cudaError_t run(const Args &p, cudaStream_t st) {
  auto blocks = [](int64_t warps) { return (unsigned)((warps + 7) / 8); };
  if (p.wr) router_kernel<T><<<blocks((int64_t)p.T * p.E), 256, 0, st>>>(p);
  route_kernel<<<p.T, 32, 0, st>>>(p);
  up_kernel<T><<<blocks((int64_t)p.T * p.k * p.I), 256, 0, st>>>(p);
  down_kernel<T><<<blocks((int64_t)p.T * p.H), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace few_tokens

size_t few_tokens_workspace(int tokens, int inter, int topk) { return (size_t)tokens * topk * inter * 4; }

cudaError_t launch_few_tokens(const sym_few_tokens &a, int, cudaStream_t st) {
  using namespace few_tokens;
  auto half = [](const void *p) { return reinterpret_cast<const uint16_t *>(p); };
  const Args p{half(a.x), half(a.w_gate), half(a.w_up), half(a.w_down), half(a.w_router), a.logits, a.idx, a.w,
               reinterpret_cast<uint16_t *>(a.out), reinterpret_cast<float *>(a.work), a.ld_x, a.ld_out, a.gate_group, a.gate_ld,
               a.up_group, a.up_ld, a.down_group, a.down_ld, a.router_ld, a.tokens, a.hidden, a.inter, a.num_experts, a.topk};
  return a.dtype == SYM_FP16 ? run<__half>(p, st) : run<__nv_bfloat16>(p, st);
}

}  // namespace symmoe
