// rows_dev.cuh -- device helpers of the row-wise kernels (SwiGLU of expert
// rows, dropout, norms around a block): element types, 16-byte vectors, the
// counter-based random words, sums over a block.
#pragma once

#include <cuda_fp16.h>
#include <cuda_bf16.h>

#include "symmoe_dev.cuh"

namespace symmoe {
namespace rows {

// VEC elements of T make one 16-byte vector
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

// V consecutive elements as floats: one 16-byte access when V is the vector
// length, one element when V is 1
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void load(const T *p, float (&f)[V]) {
  const Pack<T, V> k = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = Elem<T>::get(k.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float (&f)[V]) {
  Pack<T, V> k;
#pragma unroll
  for (int i = 0; i < V; ++i) k.v[i] = Elem<T>::put(f[i]);
  *reinterpret_cast<Pack<T, V> *>(p) = k;
}

// Columns [c, c + V) of a row, of which those outside [0, cols) do not exist
// (zeros on a load, skipped on a store); whole vectors are 16-byte accesses,
// so c places p + c on a 16-byte boundary.
template <typename T, int V>
__device__ __forceinline__ void load_part(const T *p, int c, int cols, float (&f)[V]) {
  if (c >= 0 && c + V <= cols) {
    load<T, V>(p + c, f);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = c + i >= 0 && c + i < cols ? Elem<T>::get(p[c + i]) : 0.f;
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T *p, int c, int cols, const float (&f)[V]) {
  if (c >= 0 && c + V <= cols) {
    store<T, V>(p + c, f);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i >= 0 && c + i < cols) p[c + i] = Elem<T>::put(f[i]);
}

// ---------------------------------------------------------------------------
// Counter-based random words: Philox 4x32 with 10 rounds (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  Block
// b of the stream (seed, offset) is the cipher of the counter
// (b mod 2^32, b >> 32, offset mod 2^32, offset >> 32) under the key
// (seed mod 2^32, seed >> 32); word j of it belongs to element 4b + j.
// ---------------------------------------------------------------------------
struct Random {
  uint64_t seed, offset;
  uint32_t threshold;  // an element is kept where its word >= threshold
  float keep_scale;    // 1 / (1 - p)
};
__device__ __forceinline__ uint4 random_block(const Random &r, uint64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
  uint32_t c2 = (uint32_t)r.offset, c3 = (uint32_t)(r.offset >> 32);
  uint32_t k0 = (uint32_t)r.seed, k1 = (uint32_t)(r.seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}
// keep factors (0 or 1 / (1 - p)) of the V elements from element `at` on
template <int V>
__device__ __forceinline__ void keep_factors(const Random &r, uint64_t at, float (&k)[V]) {
  if (V >= 4 && (at & 3u) == 0) {  // whole blocks
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const uint4 w = random_block(r, (at + i) >> 2);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4 && i + j < V; ++j) k[i + j] = u[j] >= r.threshold ? r.keep_scale : 0.f;
    }
    return;
  }
  uint64_t have = ~0ull;
  uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint64_t b = (at + i) >> 2;
    if (b != have) {
      w = random_block(r, b);
      have = b;
    }
    const uint32_t j = (uint32_t)(at + i) & 3u;
    const uint32_t u = j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w;
    k[i] = u >= r.threshold ? r.keep_scale : 0.f;
  }
}

// ---------------------------------------------------------------------------
// Sums of K values over the `warps` warps of a row group; every thread gets
// the totals, added in a fixed order.  buf holds 2 * 32 * K floats per group;
// `turn` alternates its halves, so one block barrier per call is enough.
// ---------------------------------------------------------------------------
template <int K>
__device__ __forceinline__ void warp_sums(float (&v)[K]) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], s);
}
template <int K>
__device__ __forceinline__ void group_sums(float (&v)[K], float *buf, int warp, int warps, int &turn) {
  warp_sums<K>(v);
  if (warps == 1) return;
  float *b = buf + turn * 32 * K;
  turn ^= 1;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) b[warp * K + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane < warps ? b[lane * K + k] : 0.f;
  warp_sums<K>(v);
}

}  // namespace rows
}  // namespace symmoe
